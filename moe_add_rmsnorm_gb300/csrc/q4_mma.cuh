// Products of 4-bit weights with several activation rows on the tensor cores (tcgen05): the projection, and a chunk's
// experts (each expert's weights with the rows that chose it: gate-up with SwiGLU, and down-and-combine).
//
// What is exact, and what is summed where: q4.cuh.  A tile is 128 weight rows (gate-up: 64 gate rows and the 64 up rows beside
// them) by up to TN activation rows.  For every 32-value block (a whole scale group, if the activation is f32 and a row has
// one unit) the tensor cores add up words times parts, an activation's two parts one after the other, into a buffer of
// tensor memory; from there the dots are scaled into f32 sums in registers.  So weights are unpacked once for all rows, and
// the tensor cores see small integers, never rounded weights.
//
// A first launch lays the activation rows out as operands: slot by slot in the order of the experts' lists, eight slots
// together, so that a chunk (four blocks) of eight slots is one contiguous copy.  In the second, one CTA an SM takes
// (expert, tile) items in turn, its warps in four roles joined by barriers of shared memory that run on from item to item:
//   0-7    unpack: four warps take the even chunks, four the odd ones; a lane is a row, whose words it turns into an operand
//          in tensor memory (from shared memory a product of 128 rows by 16 values takes 40 cycles however few its columns;
//          from there it takes 16 up to 32 columns, 32 for 64)
//   8-15   read back: a lane is a row of the tile (its warp's quarter of tensor memory), for half of the columns
//   16     issues the products
//   17     copies the activations' chunks, 18 the weights', two at a time (rows of 128 bytes)
// What bounds it is the chunks' way through the roles (950 to 1450 cycles for 128 rows by 128 values, of which an f32 row's
// products are 256 up to 32 columns) and an item's start and end.  Measured, replayed: 200 f32 rows by 6 of 64 experts of
// 2048 x 1408 190 us (295 MB; 43 at the measured copy rate), 61 f32 rows by 8192 x 4096 23 (21 MB; 3.1).  With the read-back
// in one set of four warps it was slower: the loads from tensor memory and the scaling are the longest role.
// Every wait is bounded; one that gives up ends the CTA in order, with what is in flight waited for, and is recorded in the
// workspace, on which such calls write nothing until q8_workspace_check.
#pragma once
#include <cuda.h>

#include "ffn4.h"
#include "q4.cuh"
#include "stream.cuh"
#include "tcgen05.cuh"

namespace q8 {

constexpr int kMmaThreads = 19 * 32;
constexpr int kRaw = 4;         // pairs of chunks of weights on their way (16 KB each)
constexpr int kOperands = 3;    // unpacked chunks in tensor memory (64 columns each)
constexpr int kScaleSlots = 8;  // chunks whose scales are held, until they are read back (see there)
constexpr int kItems = 32;      // items a CTA looks up at its start
constexpr unsigned kMmaPolls = 1u << 20;

struct MmaParams {
    Q4View w0, w1;
    Q4Act act;
    int kind;
    int64_t E, out_rows;
    int R, K;
    int64_t slots;       // DENSE: rows; else bound by the choices and eight a group
    PlanPtrs plan;
    const int32_t* ids;
    char* parts;         // [chunks][slots / 8][part][16][8][16 bytes]: a chunk of a tile's columns is one piece
    float* scales;       // f32: [slots], a row's unit; words: [chunks][slots / 8][4][8]
    float* y;
    int64_t y_stride;
    float* out;          // down: [R * K][out_rows]
    int chunks, row_tiles, col_tiles;  // col_tiles: the projection's
    int slices;          // parts of the columns of weights (the projection's; their sums meet in `sums`)
    float* sums;         // [tiles][slices][TN][128]
    int* counters;       // [tiles], zero between calls
    int* failed;
};

// An expert's rows: its place in the lists and the slots they are laid out in.
struct Group {
    int e, first, count, slot;  // e < 0: none
};

// The products' kernel reads the plan and the workspace's word before its dependency wait, as do the warps' products (q4_rows.cuh).
// Only the launch that lays the rows out comes between, and it lets this one start after its own wait has returned in every
// CTA: what earlier launches wrote is in L2 by then, and an SM's L1 keeps no line from before a launch's start.  Loads that pass
// L1 by would say so without that second step, and took a chunk's experts from 190 to 192.5 us.
__device__ __forceinline__ int mma_groups(const MmaParams& p) {
    if (p.kind == Q4_DENSE) return 1;
    return min(max(p.plan.active[0], 0), (int)min(p.E, (int64_t)p.R * p.K));
}

// Where expert e's slots start, its rows standing from place `first` of the lists on: a multiple of eight, and with at most seven
// lost an expert no two experts' meet.
__device__ __forceinline__ int mma_slot(int first, int e) { return (first + 7 * e + 7) & ~7; }

// Group a.
__device__ __forceinline__ Group mma_group(const MmaParams& p, int a) {
    if (p.kind == Q4_DENSE) return Group{0, 0, p.R, 0};
    Group g;
    const int total = p.R * p.K;
    g.e = p.plan.active[1 + a];
    if (g.e < 0 || g.e >= p.E) return Group{-1, 0, 0, 0};
    g.first = min(max(p.plan.offsets[g.e], 0), total);
    g.count = max(min(p.plan.offsets[g.e + 1], total) - g.first, 0);
    g.slot = mma_slot(g.first, g.e);
    return g;
}

// The choice at place i of the lists (-1: none).
__device__ __forceinline__ int mma_choice(const MmaParams& p, int i) {
    if (p.kind == Q4_DENSE) return i;
    const int c = p.plan.lists[i];
    return c >= 0 && c < p.R * p.K ? c : -1;
}

// Lays out one slot at a time: row r of the projection, or the row of the choice at place r of the lists.
template <int FORM>
__global__ void __launch_bounds__(256) q4_slots_kernel(const MmaParams p) {
    constexpr int PARTS = FORM == FORM_ONE ? 1 : 2;
    __shared__ float most[2][8];
    __shared__ int where[2];
    griddep_wait();    // the launch before has ended, which the products' launch takes for granted from its start on
    griddep_launch();
    const int octets = 16 * p.chunks, cols = p.w0.cols, lane = threadIdx.x & 31;
    const int n = p.kind == Q4_DENSE ? p.R : p.R * p.K;
    int buf = 0;
    for (int i = blockIdx.x; i < n; i += gridDim.x, buf ^= 1) {
        int c = i, slot = i;
        if (p.kind != Q4_DENSE) {
            if (threadIdx.x == 0) {
                c = mma_choice(p, i);
                slot = -1;
                const int e = c >= 0 ? p.ids[c] : -1;
                if (e >= 0 && e < p.E) {
                    const int first = p.plan.offsets[e];
                    if (first >= 0 && i >= first && i < p.plan.offsets[e + 1]) slot = mma_slot(first, e) + i - first;
                }
                if (slot >= p.slots) slot = -1;
                where[0] = c, where[1] = slot;
            }
            __syncthreads();
            c = where[0], slot = where[1];
            __syncthreads();
            if (slot < 0) continue;
        }
        const int64_t r = p.kind == Q4_GATE_UP ? c / p.K : c;
        float m = 0.f;
        if (FORM == FORM_F32) {
            for (int o = threadIdx.x; o < octets; o += blockDim.x) {
                float x[8];
                act_values(p.act, r, o, cols, x);
                m = fmaxf(m, finite_max(x));
            }
            m = warp_max(m);
            if (lane == 0) most[buf][threadIdx.x >> 5] = m;
            __syncthreads();
            for (int k = 0; k < 8; ++k) m = fmaxf(m, most[buf][k]);
        }
        for (int o = threadIdx.x; o < octets; o += blockDim.x) {
            const int64_t chunk = (int64_t)(o >> 4) * (p.slots >> 3) + (slot >> 3);
            ActParts a;
            if (FORM == FORM_F32) {
                float x[8];
                act_values(p.act, r, o, cols, x);
                a = split_values(x, m);
                if (o == 0) p.scales[slot] = a.scale;
            } else {
                a = act_words(p.act, r, o, cols);
                if ((o & 3) == 0) p.scales[chunk * 32 + ((o >> 2) & 3) * 8 + (slot & 7)] = a.scale;
            }
            char* at = p.parts + chunk * (PARTS * 2048) + (o & 15) * 128 + (slot & 7) * 16;
            *reinterpret_cast<uint4*>(at) = a.hi;
            if (PARTS == 2) *reinterpret_cast<uint4*>(at + 2048) = a.lo;
        }
    }
}

// Descriptor of a K-major operand without swizzle at shared address `at`: core matrices of 8 rows x 16 bytes, `lbo` bytes apart
// along K and `sbo` bytes apart along the rows.
__device__ __forceinline__ uint64_t operand_desc(uint32_t at, uint32_t lbo, uint32_t sbo) {
    return (uint64_t)((at >> 4) & 0x3FFF) | ((uint64_t)((lbo >> 4) & 0x3FFF) << 16) | ((uint64_t)((sbo >> 4) & 0x3FFF) << 32) |
           (1ull << 46);
}

// Whether this lane is the one of the converged warp that issues products and commits: the compiler then keeps their operands
// in uniform registers (from `lane == 0` every operand of every product took moves of its own: 340 cycles a product).
__device__ __forceinline__ bool elected() {
    uint32_t q;
    asm volatile("{ .reg .pred q; elect.sync _|q, 0xffffffff; selp.u32 %0, 1, 0, q; }" : "=r"(q));
    return q != 0;
}

// D[tmem] (+)= A B for 16 values, A in tensor memory.
__device__ __forceinline__ void tc_mma_ta(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile("{ .reg .pred p; setp.ne.u32 p, %4, 0; tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p; }" ::"r"(d), "r"(a),
                 "l"(b), "r"(idesc), "r"(acc));
}

// Columns of this warp's 32 lanes of tensor memory: read (complete after tc_wait_ld), and written (after tmem_wait_store).
__device__ __forceinline__ void tmem_load(uint32_t at, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(at));
}
__device__ __forceinline__ void tmem_load(uint32_t at, uint32_t (&r)[16]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
                   "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                 : "r"(at));
}
__device__ __forceinline__ void tmem_load(uint32_t at, uint32_t (&r)[32]) { tc_ld32(at, r); }
// After tc_wait_ld, for each load's registers: nothing that reads them moves above the wait.
template <int N>
__device__ __forceinline__ void tmem_loaded(uint32_t (&r)[N]) {
#pragma unroll
    for (int i = 0; i < N; i += 8)
        asm volatile("" : "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), "+r"(r[i + 4]), "+r"(r[i + 5]), "+r"(r[i + 6]),
                          "+r"(r[i + 7])::"memory");
}
__device__ __forceinline__ void tmem_store(uint32_t at, const uint32_t (&r)[4][4]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(at),
                 "r"(r[0][0]), "r"(r[0][1]), "r"(r[0][2]), "r"(r[0][3]), "r"(r[1][0]), "r"(r[1][1]), "r"(r[1][2]), "r"(r[1][3]),
                 "r"(r[2][0]), "r"(r[2][1]), "r"(r[2][2]), "r"(r[2][3]), "r"(r[3][0]), "r"(r[3][1]), "r"(r[3][2]), "r"(r[3][3])
                 : "memory");
}
__device__ __forceinline__ void tmem_wait_store() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// A box of the map's bytes, from byte x of row y on, into shared memory, counted on `bar`.
__device__ __forceinline__ void tile_g2s(void* dst, const CUtensorMap* map, int x, int y, uint64_t* bar) {
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
                 ::"r"(smem_addr(dst)), "l"(map), "r"(x), "r"(y), "r"(smem_addr(bar))
                 : "memory");
}

// The rest of a wait whose first poll found its phase open, by one lane or a whole warp: false when it gave up, or when another of
// the CTA's did.
static __device__ __noinline__ bool mma_wait_on(uint64_t* bar, unsigned parity, int* dead, int* failed) {
    for (unsigned i = 0; i < kMmaPolls; ++i) {
        if (mbar_try_wait(bar, parity & 1u)) return true;
        if (*(volatile int*)dead) return false;
        if (i > 64) __nanosleep(32);
    }
    *(volatile int*)dead = 1;
    atomicExch(failed, 1);
    return false;
}

template <int FORM, int TN>
struct MmaShared {
    static constexpr int PARTS = FORM == FORM_ONE ? 1 : 2;
    static constexpr int kColumns = TN == 64 ? 3 : 4;         // chunks of activations on their way
    alignas(1024) char raw[kRaw][128 * 128];                  // [128 rows][128 bytes], 16-byte units swizzled by row % 8
    alignas(128) char b[kColumns][TN / 8][PARTS][16][128];    // [eight slots][part][along K]
    float wscale[kScaleSlots][4][128];
    float cscale[FORM == FORM_F32 ? 1 : kScaleSlots][TN / 8][4][8];
    float sums[TN][128], unit[TN];                            // a tile's results
    int choice[TN];
    uint64_t raw_full[kRaw], raw_empty[kRaw], a_full[kOperands], a_empty[kOperands], b_full[kColumns], b_empty[kColumns];
    uint64_t s_full[kScaleSlots], c_full[kScaleSlots], t_full[8], t_empty[8], ready, drain;
    Group groups[kItems];
    uint32_t tmem;
    int dead, last;
};

template <int FORM, int TN>
__global__ void __launch_bounds__(kMmaThreads, 1) q4_mma_kernel(const __grid_constant__ MmaParams p,
                                                               const __grid_constant__ CUtensorMap map0,
                                                               const __grid_constant__ CUtensorMap map1) {
    constexpr int PARTS = FORM == FORM_ONE ? 1 : 2;
    constexpr int kColumns = MmaShared<FORM, TN>::kColumns;
    constexpr int kSums = kOperands * 64;  // the dots' buffers start at this column of tensor memory
    extern __shared__ __align__(1024) char smem[];
    auto& sh = *reinterpret_cast<MmaShared<FORM, TN>*>(smem);
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    griddep_launch();
    const bool gate_up = p.kind == Q4_GATE_UP;
    const int nb = p.w0.cols >> 5, tile_rows = gate_up ? 64 : 128, last_row = (int)p.out_rows - 1;
    // Blocks whose dots share a buffer; buffers that are handed over together (a hand-over costs the warps 100 cycles and
    // more on either side: a chunk's buffers, or half of them where tensor memory holds no more); and such sets.
    const int unit_log2 = FORM == FORM_F32 ? p.w0.group_log2 - 5 : 0, unit = 1 << unit_log2, units = 4 >> unit_log2;
    const int set = min(units, TN == 64 ? 2 : 4), sets = set == 4 || TN == 64 ? 2 : 4;  // (set * sets * TN: at most 256 columns)
    const int per_group = p.row_tiles * p.col_tiles * p.slices;
    const int items = mma_groups(p) * per_group;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kRaw; ++i) mbar_init(&sh.raw_full[i], 1), mbar_init(&sh.raw_empty[i], 8);
        for (int i = 0; i < kOperands; ++i) mbar_init(&sh.a_full[i], 4), mbar_init(&sh.a_empty[i], 1);
        for (int i = 0; i < kColumns; ++i) mbar_init(&sh.b_full[i], 1), mbar_init(&sh.b_empty[i], 1);
        for (int i = 0; i < kScaleSlots; ++i) mbar_init(&sh.s_full[i], 4), mbar_init(&sh.c_full[i], 1);
        for (int i = 0; i < 8; ++i) mbar_init(&sh.t_full[i], 1), mbar_init(&sh.t_empty[i], 8);
        mbar_init(&sh.ready, 1);
        mbar_init(&sh.drain, 1);
        fence_barrier_init();
        sh.dead = *p.failed;  // (an earlier call's wait gave up: its counters may not be zero)
    }
    if (threadIdx.x < kItems) {
        const int item = blockIdx.x + threadIdx.x * gridDim.x;
        if (item < items) sh.groups[threadIdx.x] = mma_group(p, item / per_group);
    }
    __syncthreads();
    bool ok = sh.dead == 0;
    // Waits of a whole warp, whose `ok` stays alike: the first polls go out together, and one vote ends them (with a branch of
    // every lane's own a wait for what was there already took 100 cycles for 30).
    auto wait3 = [&](uint64_t* x, unsigned px, uint64_t* y, unsigned py, uint64_t* z, unsigned pz) {
        const bool bx = mbar_try_wait(x, px & 1u), by = mbar_try_wait(y, py & 1u), bz = mbar_try_wait(z, pz & 1u);
        if (__all_sync(0xffffffffu, (bx && by && bz) || !ok)) return;
        ok = __all_sync(0xffffffffu, mma_wait_on(x, px, &sh.dead, p.failed) && mma_wait_on(y, py, &sh.dead, p.failed) &&
                                         mma_wait_on(z, pz, &sh.dead, p.failed));
    };
    auto wait2 = [&](uint64_t* x, unsigned px, uint64_t* y, unsigned py) {
        const bool bx = mbar_try_wait(x, px & 1u), by = mbar_try_wait(y, py & 1u);
        if (__all_sync(0xffffffffu, (bx && by) || !ok)) return;
        ok = __all_sync(0xffffffffu, mma_wait_on(x, px, &sh.dead, p.failed) && mma_wait_on(y, py, &sh.dead, p.failed));
    };
    auto wait = [&](uint64_t* x, unsigned px) {
        if (__all_sync(0xffffffffu, mbar_try_wait(x, px & 1u) || !ok)) return;
        ok = __all_sync(0xffffffffu, mma_wait_on(x, px, &sh.dead, p.failed));
    };
    // When the CTA ends nothing may be on its way into shared memory: a role that copies or multiplies waits for the last of
    // its own, which the role that uses them may have given up on.
    auto drain = [&](uint64_t* x, unsigned px) {
        for (unsigned n = 0; n < 1024 && !mbar_try_wait(x, px & 1u); ++n) __nanosleep(64);
    };
    auto wait_one = [&](uint64_t* x, unsigned px) { ok = ok && mma_wait_on(x, px, &sh.dead, p.failed); };  // of one lane
    // Item k of the CTA: group, tile of rows, first and last tile of columns, chunks.  (The experts' items take all their
    // columns, the weights once for each tile of them.)
    struct Item {
        Group g;
        int row_tile, ct, cts, c0, c1;
    };
    auto item_at = [&](int k, Item& it) {
        const int item = blockIdx.x + k * gridDim.x;
        if (item >= items) return false;
        it.g = k < kItems ? sh.groups[k] : mma_group(p, item / per_group);
        int rest = item % per_group;
        const int slice = rest % p.slices;
        rest /= p.slices;
        it.row_tile = rest % p.row_tiles;
        const int all = it.g.e < 0 ? 0 : (it.g.count + TN - 1) / TN;
        it.ct = p.kind == Q4_DENSE ? rest / p.row_tiles : 0;
        it.cts = p.kind == Q4_DENSE ? it.ct + 1 : all;
        it.c0 = (int)((int64_t)p.chunks * slice / p.slices);
        it.c1 = (int)((int64_t)p.chunks * (slice + 1) / p.slices);
        return true;
    };
    auto columns = [&](const Item& it) { return min(it.g.count - it.ct * TN, TN); };

    if (w < 8) {
        // ---- unpack ------------------------------------------------------------------------------------------------------
        const int r = 32 * (w & 3) + lane, odd = w >> 2;
        const int row_groups = p.w0.cols >> p.w0.group_log2, per_chunk = 4 / (1 << (p.w0.group_log2 - 5));
        const bool second = gate_up && r >= 64;
        const Q4View& v = second ? p.w1 : p.w0;
        // a chunk's scales (and zero points) in one load, where every row's stand at a multiple of their size
        const bool wide = row_groups % per_chunk == 0 && ((uintptr_t)v.s % (2 * per_chunk)) == 0 && ((uintptr_t)v.z % per_chunk) == 0;
        uint32_t s[4], z[4];
        int64_t sg = 0;
        auto scales = [&](int c) {
            const int64_t at = sg + (int64_t)c * per_chunk;
            if (wide) {
                if (per_chunk == 4) {
                    const uint2 u = __ldg(reinterpret_cast<const uint2*>(v.s + at));
                    s[0] = u.x, s[1] = u.y;
                    if (v.z) z[0] = __ldg(reinterpret_cast<const uint32_t*>(v.z + at));
                } else if (per_chunk == 2) {
                    s[0] = __ldg(reinterpret_cast<const uint32_t*>(v.s + at));
                    if (v.z) z[0] = __ldg(reinterpret_cast<const uint16_t*>(v.z + at));
                } else {
                    s[0] = __ldg(v.s + at);
                    if (v.z) z[0] = __ldg(v.z + at);
                }
                return;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const bool in = i < per_chunk && c * per_chunk + i < row_groups;
                s[i] = in ? __ldg(v.s + at + i) : 0u;
                z[i] = in && v.z ? __ldg(v.z + at + i) : 8u;
            }
        };
        // This warp's next chunk: every other one of a tile of columns, from c on; its number among all the CTA's chunks and the
        // number of its pair.
        Item it;
        int k = 0, c = 0, again = 0;
        unsigned gi = 0, pair = 0, tile_gi = 0, tile_pair = 0;
        bool left = true;
        auto next_tile = [&]() {
            if (again > 0) {  // the same weights for the next columns
                --again;
                return;
            }
            do {
                left = item_at(k++, it);
                if (!left) return;
            } while (it.ct >= it.cts || it.c0 >= it.c1);
            again = it.cts - it.ct - 1;
            const int row = min(it.row_tile * tile_rows + (second ? r - 64 : r), last_row);
            sg = ((int64_t)it.g.e * p.out_rows + row) * row_groups;
        };
        auto settle = [&]() {  // c is past the tile's end: the next tile that has a chunk for this warp
            while (left && c >= it.c1) {
                tile_gi += it.c1 - it.c0;
                tile_pair += (it.c1 - it.c0 + 1) >> 1;
                next_tile();
                c = it.c0 + odd;
            }
            gi = tile_gi + (c - it.c0);
            pair = left ? tile_pair + ((c - it.c0) >> 1) : tile_pair;
        };
        wait(&sh.ready, 0);
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        const uint32_t tmem = sh.tmem + ((uint32_t)(32 * (w & 3)) << 16);
        const uint32_t row_at = r * 128 + odd * 64, swizzle = r & 7;
        next_tile();
        if (left) c = it.c0 + odd;
        settle();
        if (left) scales(c);
        for (unsigned done = 0;; ++done) {
            for (; done < pair; ++done) {  // pairs without a chunk for this warp
                wait(&sh.raw_full[done % kRaw], done / kRaw);
                if (lane == 0 && ok) mbar_arrive(&sh.raw_empty[done % kRaw]);
            }
            if (!left) break;
            const int slot = gi % kScaleSlots, stage = gi % kOperands, from = pair % kRaw;
            const unsigned stage_phase = gi / kOperands, from_phase = pair / kRaw;
            float sw[4];
            uint32_t zc[4];
            if (wide && per_chunk == 1) {
                sw[0] = sw[1] = sw[2] = sw[3] = scale_f32(s[0], p.w0.bf16);
            } else if (wide && per_chunk == 2) {
                sw[0] = sw[1] = scale_f32(s[0] & 0xffffu, p.w0.bf16);
                sw[2] = sw[3] = scale_f32(s[0] >> 16, p.w0.bf16);
            } else {
                if (wide) s[3] = s[1] >> 16, s[2] = s[1] & 0xffffu, s[1] = s[0] >> 16, s[0] = s[0] & 0xffffu;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int i = (j * per_chunk) >> 2;
                    sw[j] = scale_f32(i == 0 ? s[0] : i == 1 ? s[1] : i == 2 ? s[2] : s[3], p.w0.bf16);
                }
            }
            if (v.z) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int i = (j * per_chunk) >> 2;
                    const uint32_t zb = wide ? (z[0] >> (8 * i)) & 0xffu : i == 0 ? z[0] : i == 1 ? z[1] : i == 2 ? z[2] : z[3];
                    zc[j] = 0x64006400u | (zb * 0x10001u);
                }
            } else {
                zc[0] = zc[1] = zc[2] = zc[3] = 0x64086408u;
            }
            c += 2;
            settle();
            if (left) scales(c);  // for this warp's next chunk
            // (the phase before a barrier's first is complete)
            wait2(&sh.raw_full[from], from_phase, &sh.a_empty[stage], stage_phase + 1);
            if (!ok) continue;
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            uint4 words[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                words[j] = *reinterpret_cast<const uint4*>(sh.raw[from] + ((row_at + 16 * j) ^ (swizzle << 4)));
#pragma unroll
            for (int j = 0; j < 4; ++j) {  // (blocks past the last are zeros in the copy, and no product reads them)
                const uint32_t zf = zero_less(zc[j]);
                uint32_t h[4][4];
                words_f16(words[j].x, zc[j], zf, h[0]);
                words_f16(words[j].y, zc[j], zf, h[1]);
                words_f16(words[j].z, zc[j], zf, h[2]);
                words_f16(words[j].w, zc[j], zf, h[3]);
                tmem_store(tmem + stage * 64 + j * 16, h);
                sh.wscale[slot][j][r] = sw[j];
            }
            tmem_wait_store();
            asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.a_full[stage]), mbar_arrive(&sh.s_full[slot]), mbar_arrive(&sh.raw_empty[from]);
        }
    } else if (w == 17) {
        // ---- the activations' copies -------------------------------------------------------------------------------------
        if (lane == 0) {
            griddep_wait();
            unsigned gi = 0;
            Item it;
            for (int k = 0; item_at(k, it); ++k) {
                if (it.c0 >= it.c1) continue;
                for (; it.ct < it.cts; ++it.ct) {
                    const int groups = (columns(it) + 7) >> 3;
                    const int64_t eight = (it.g.slot + it.ct * TN) >> 3;
                    for (int c = it.c0; c < it.c1 && ok; ++c, ++gi) {
                        const int stage = gi % kColumns, slot = gi % kScaleSlots;
                        if (gi >= kColumns) wait_one(&sh.b_empty[stage], gi / kColumns - 1);
                        if (!ok) break;
                        const int64_t chunk = c * (p.slots >> 3) + eight;
                        mbar_arrive_expect_tx(&sh.b_full[stage], groups * PARTS * 2048);
                        bulk_g2s(sh.b[stage], p.parts + chunk * (PARTS * 2048), groups * PARTS * 2048, &sh.b_full[stage]);
                        if (FORM != FORM_F32) {
                            mbar_arrive_expect_tx(&sh.c_full[slot], groups * 128);
                            bulk_g2s(sh.cscale[FORM == FORM_F32 ? 0 : slot], p.scales + chunk * 32, groups * 128, &sh.c_full[slot]);
                        }
                    }
                }
            }
            for (unsigned i = gi > kColumns ? gi - kColumns : 0; i < gi; ++i) drain(&sh.b_full[i % kColumns], i / kColumns);
            for (unsigned i = gi > kScaleSlots ? gi - kScaleSlots : 0; i < gi && FORM != FORM_F32; ++i)
                drain(&sh.c_full[i % kScaleSlots], i / kScaleSlots);
        }
    } else if (w == 18) {
        // ---- the weights' copies -----------------------------------------------------------------------------------------
        if (lane == 0) {
            unsigned pair = 0;
            Item it;
            for (int k = 0; item_at(k, it); ++k) {
                if (it.c0 >= it.c1) continue;
                const int row = (int)((int64_t)it.g.e * p.out_rows) + it.row_tile * tile_rows;
                for (; it.ct < it.cts; ++it.ct)
                    for (int c = it.c0; c < it.c1 && ok; c += 2, ++pair) {
                        const int to = pair % kRaw;
                        if (pair >= kRaw) wait_one(&sh.raw_empty[to], pair / kRaw - 1);
                        if (!ok) break;
                        mbar_arrive_expect_tx(&sh.raw_full[to], 128 * 128);
                        tile_g2s(sh.raw[to], &map0, 64 * c, row, &sh.raw_full[to]);
                        if (gate_up) tile_g2s(sh.raw[to] + 64 * 128, &map1, 64 * c, row, &sh.raw_full[to]);
                    }
            }
            for (unsigned i = pair > kRaw ? pair - kRaw : 0; i < pair; ++i) drain(&sh.raw_full[i % kRaw], i / kRaw);
        }
    } else if (w == 16) {
        // ---- the products -----------------------------------------------------------------------------------------------
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(&sh.tmem)));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
        __syncwarp();
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        const uint32_t tmem = sh.tmem;
        if (lane == 0) mbar_arrive(&sh.ready);
        const uint64_t b0 = operand_desc(smem_addr(sh.b[0]), 128, PARTS * 2048);
        unsigned gi = 0, ui = 0;
        int stage = 0, buf = 0;
        Item it;
        for (int k = 0; item_at(k, it); ++k) {
            if (it.c0 >= it.c1) continue;
            for (; it.ct < it.cts; ++it.ct) {
                const uint32_t idesc = tc_idesc_f16(128, (columns(it) + 15) & ~15);
                for (int c = it.c0; c < it.c1; ++c, ++gi) {
                    wait3(&sh.a_full[stage], gi / kOperands, &sh.b_full[gi % kColumns], gi / kColumns, &sh.t_empty[buf], ui / sets + 1);
                    const uint64_t b = b0 + (gi % kColumns) * (TN / 8 * PARTS * 2048 >> 4);
                    const uint32_t a = tmem + stage * 64;
                    for (int u = 0; u < units; u += set, ++ui) {  // (a last chunk's missing units keep their buffers)
                        if (u > 0) wait(&sh.t_empty[buf], ui / sets + 1);
                        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                        const int first = u << unit_log2, end = min((u + set) << unit_log2, nb - 4 * c);
                        const uint32_t d = tmem + kSums + buf * set * TN;
                        if (elected() && ok) {
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                if (j < first || j >= end) continue;
                                const uint32_t dj = d + ((j - first) >> unit_log2) * TN;
                                tc_mma_ta(dj, a + j * 16, b + j * 32, idesc, j & (unit - 1));
                                tc_mma_ta(dj, a + j * 16 + 8, b + j * 32 + 16, idesc, 1);
                                if (PARTS == 2) {  // the second part's operand stands 2048 bytes on
                                    tc_mma_ta(dj, a + j * 16, b + j * 32 + 128, idesc, 1);
                                    tc_mma_ta(dj, a + j * 16 + 8, b + j * 32 + 144, idesc, 1);
                                }
                            }
                            tc_commit(&sh.t_full[buf]);
                            if (u + set >= units) tc_commit(&sh.a_empty[stage]), tc_commit(&sh.b_empty[gi % kColumns]);
                        }
                        __syncwarp();
                        buf = buf == sets - 1 ? 0 : buf + 1;
                    }
                    stage = stage == kOperands - 1 ? 0 : stage + 1;
                }
            }
        }
        if (elected()) tc_commit(&sh.drain);  // (no product may be under way when its operands and its tensor memory go)
        __syncwarp();
        drain(&sh.drain, 0);
        __syncwarp();
    } else {
        // ---- read back -----------------------------------------------------------------------------------------------
        // A chunk's scales are overwritten kScaleSlots chunks on.  Chunk c's are written once the products of c - kOperands are
        // done (copied: of c - kColumns), and these started once the reading had given back the buffers they use, which are
        // those of `sets` sets before: of four chunks at most (an f32 row's groups of 64 and 128; words have two).  The
        // reading gives a buffer back only after it has used the scales of all before it, so chunk c - 7's have been used.
        static_assert(kScaleSlots >= kOperands + 4 && kScaleSlots >= kColumns + 2, "scales in use are not overwritten");
        static_assert(kSums + 256 <= 512, "the operands' and the dots' columns of tensor memory");
        const int r = 32 * (w & 3) + lane;
        constexpr int HN = TN / 2;
        const int col0 = w >= 12 ? HN : 0;
        auto sync = [&]() { asm volatile("bar.sync 1, 256;" ::: "memory"); };
        wait(&sh.ready, 0);
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        const uint32_t tmem = sh.tmem + ((uint32_t)(32 * (w & 3)) << 16) + kSums + col0;
        griddep_wait();  // (the rows' units)
        unsigned gi = 0, ui = 0;
        int buf = 0;
        Item it;
        for (int k = 0; item_at(k, it); ++k) {
            if (it.c0 >= it.c1) continue;
            for (; it.ct < it.cts; ++it.ct) {
                const int n = columns(it), place = it.g.first + it.ct * TN;
                // thread j: column j's choice and unit, looked at only at the end (a wait for them here held up the first chunk)
                int choice = place + r;
                float column_unit = 1.f;
                if (col0 == 0 && r < n) {
                    if (p.kind != Q4_DENSE) choice = p.plan.lists[place + r];
                    if (FORM == FORM_F32) column_unit = p.scales[it.g.slot + it.ct * TN + r];
                }
                float2 acc[HN / 2] = {};
                for (int c = it.c0; c < it.c1; ++c, ++gi) {
                    const int slot = gi % kScaleSlots;
                    if (FORM == FORM_F32) wait2(&sh.s_full[slot], gi / kScaleSlots, &sh.t_full[buf], ui / sets);
                    else wait3(&sh.s_full[slot], gi / kScaleSlots, &sh.c_full[slot], gi / kScaleSlots, &sh.t_full[buf], ui / sets);
                    for (int u0 = 0; u0 < units; u0 += set, ++ui) {
                        if (u0 > 0) wait(&sh.t_full[buf], ui / sets);
                        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                        __syncwarp();
                        // as many units' columns on their way together as registers hold
                        const int here = min(set, (nb - 4 * c + unit - 1) / unit - u0);
                        if (ok && here > 0 && col0 < n) {
                            constexpr int most = TN == 64 ? 2 : 4, batch = TN == 64 ? 1 : TN == 32 ? 2 : 4;
                            const uint32_t from = tmem + buf * set * TN;
#pragma unroll
                            for (int q0 = 0; q0 < most; q0 += batch) {
                                if (q0 >= here) break;
                                uint32_t d[batch][HN];
#pragma unroll
                                for (int q = 0; q < batch; ++q)
                                    if (q0 + q < here) tmem_load(from + (q0 + q) * TN, d[q]);
                                tc_wait_ld();
#pragma unroll
                                for (int q = 0; q < batch; ++q) {
                                    tmem_loaded(d[q]);
                                    if (q0 + q >= here) break;
                                    const int b = (u0 + q0 + q) << unit_log2;
                                    const float sw = sh.wscale[slot][b][r];
                                    const float2 s2 = make_float2(sw, sw);
#pragma unroll
                                    for (int i = 0; i < HN / 2; ++i) {
                                        float2 s = s2;
                                        if (FORM != FORM_F32) {
                                            const int col = col0 + 2 * i;
                                            s = pair_mul(s, *reinterpret_cast<const float2*>(
                                                                &sh.cscale[FORM == FORM_F32 ? 0 : slot][col >> 3][b][col & 7]));
                                        }
                                        pair_fma(acc[i], s, __uint_as_float(d[q][2 * i]), __uint_as_float(d[q][2 * i + 1]));
                                    }
                                }
                            }
                        }
                        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&sh.t_empty[buf]);
                        buf = buf == sets - 1 ? 0 : buf + 1;
                    }
                }
                bool write = ok;
                if (p.slices > 1) {  // this slice's sums; the last to arrive adds the slices in their order
                    const int tile = it.ct * p.row_tiles + it.row_tile;
                    const int slice = (blockIdx.x + k * gridDim.x) % p.slices;
                    float* sums = p.sums + ((int64_t)tile * p.slices) * (TN * 128) + col0 * 128 + r;
#pragma unroll
                    for (int j = 0; j < HN; ++j)
                        if (ok && col0 + j < n) __stcg(sums + slice * (TN * 128) + j * 128, j & 1 ? acc[j >> 1].y : acc[j >> 1].x);
                    __threadfence();
                    sync();
                    if (threadIdx.x == 256) sh.last = ok && atomic_add_acq_rel_gpu(p.counters + tile, 1) == p.slices - 1;
                    sync();
                    write = ok && sh.last;
                    if (write) {
                        for (int k2 = 0; k2 < p.slices; ++k2) {  // (a slice's loads on their way together)
                            float v[HN];
#pragma unroll
                            for (int j = 0; j < HN; ++j) v[j] = col0 + j < n ? __ldcg(sums + k2 * (TN * 128) + j * 128) : 0.f;
#pragma unroll
                            for (int j = 0; j < HN; ++j) {
                                float& to = j & 1 ? acc[j >> 1].y : acc[j >> 1].x;
                                to = k2 == 0 ? v[j] : to + v[j];
                            }
                        }
                        if (threadIdx.x == 256) p.counters[tile] = 0;
                    }
                }
                // The sums go through shared memory, so that short loops write them (unrolled over the columns this end took as
                // long as ten chunks).
                if (col0 == 0 && r < TN) {
                    sh.choice[r] = r < n && choice >= 0 && choice < p.R * p.K ? choice : -1;
                    sh.unit[r] = column_unit;
                }
#pragma unroll
                for (int j = 0; j < HN; ++j) sh.sums[col0 + j][r] = j & 1 ? acc[j >> 1].y : acc[j >> 1].x;
                sync();
                if (write) {
                    const int id = threadIdx.x - 256;
                    if (gate_up) {  // 64 threads a column
                        const int row = it.row_tile * 64 + (id & 63);
#pragma unroll 4
                        for (int j = id >> 6; j < n; j += 4) {
                            const int to = sh.choice[j];
                            const float u = sh.unit[j];
                            if (to >= 0 && row <= last_row)
                                p.y[to * p.y_stride + row] = silu_f32(sh.sums[j][id & 63] * u) * (sh.sums[j][64 + (id & 63)] * u);
                        }
                    } else {
                        const int row = it.row_tile * 128 + r;
#pragma unroll 4
                        for (int j = id >> 7; j < n; j += 2) {
                            const int to = sh.choice[j];
                            const float v = sh.sums[j][r] * sh.unit[j];
                            if (to >= 0 && row <= last_row) (p.kind == Q4_DENSE ? p.y + to * p.y_stride : p.out + to * p.out_rows)[row] = v;
                        }
                    }
                }
                sync();  // (the sums' place is free again)
            }
        }
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    if (w == 16) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(sh.tmem));
}

// The map of a matrix's words as rows of bytes, read in boxes of 128 bytes by box_rows (q4_several.cu).
bool q4_map(CUtensorMap* map, const Q4View& w, int box_rows);

template <int FORM, int TN>
cudaError_t run_mma(MmaParams p, int64_t groups, Carve& ws, cudaStream_t st) {
    const int sms = device_info().sms;
    p.col_tiles = p.kind == Q4_DENSE ? (p.R + TN - 1) / TN : 1;
    const int64_t tiles = (int64_t)p.row_tiles * p.col_tiles;
    p.slices = 1;
    if (p.kind == Q4_DENSE && tiles * 2 <= sms) {  // too few tiles for the SMs: four chunks a slice or more (2048 x 4096, 32 rows 22 -> 14 us)
        p.slices = (int)min(min((int64_t)sms / tiles, (int64_t)8), (int64_t)max(p.chunks / 4, 1));
        if (p.slices > 1) {
            p.sums = ws.take<float>((size_t)tiles * p.slices * TN * 128);
            p.counters = ws.take_counters((size_t)tiles);
            if (ws.overflow) return cudaSuccess;
        }
    }
    const int64_t items = groups * tiles * p.slices;
    if (items > 0x7fffffff) return cudaErrorInvalidValue;
    CUtensorMap m0, m1;
    const bool gate_up = p.kind == Q4_GATE_UP;
    if (!q4_map(&m0, p.w0, gate_up ? 64 : 128) || !q4_map(&m1, gate_up ? p.w1 : p.w0, gate_up ? 64 : 128)) return cudaErrorInvalidValue;
    const dim3 lay((unsigned)min(p.kind == Q4_DENSE ? (int64_t)p.R : (int64_t)p.R * p.K, (int64_t)sms * 8));
    cudaError_t e = launch(q4_slots_kernel<FORM>, lay, dim3(256), 0, st, 1, p);
    if (e != cudaSuccess) return e;
    constexpr size_t smem = sizeof(MmaShared<FORM, TN>);
    static_assert(smem <= 232448, "a CTA's shared memory");
    static std::atomic<uint64_t> done;
    e = allow_smem(q4_mma_kernel<FORM, TN>, smem, done);
    if (e != cudaSuccess) return e;
    return launch(q4_mma_kernel<FORM, TN>, dim3((unsigned)min(items, (int64_t)sms)), dim3(kMmaThreads), smem, st, 1, p, m0, m1);
}

template <int FORM>
cudaError_t launch_mma(const MmaParams& p, int64_t groups, Carve& ws, cudaStream_t st) {
    // Rows a tile: the projection's, or an expert's average and one and a half deviations of a random choice.  Measured, us, 16, 32
    // and 64 a tile, 6 of 64 experts of 2048 x 1408: 100 rows (9.4 an expert) 184, 199 and 276; 160 (15) 286, 211 and 282; 400 (37.5)
    // 497, 387 and 319.
    const double mean = (double)p.R * p.K / groups;
    const double rows = p.kind == Q4_DENSE ? p.R : mean + 1.5 * sqrt(mean);
    int tile = rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
    // A projection that leaves half of the SMs idle at half of that takes half: 2048 x 4096, 64 rows 17.5 and 14.7 us (64 and 32 a
    // tile), 32 rows 13.9 and 13.0 (32 and 16); with more tiles the weights' second unpacking costs more, 8192 x 4096, 64 rows 22.5
    // and 24.4.
    if (p.kind == Q4_DENSE && tile > 16 && p.row_tiles * ((p.R + tile / 2 - 1) / (int64_t)(tile / 2)) * 2 <= device_info().sms) tile /= 2;
    if (tile == 16) return run_mma<FORM, 16>(p, groups, ws, st);
    if (tile == 32) return run_mma<FORM, 32>(p, groups, ws, st);
    return run_mma<FORM, 64>(p, groups, ws, st);
}

// One file each, so that they compile beside one another.
cudaError_t launch_mma_f32(const MmaParams& p, int64_t groups, Carve& ws, cudaStream_t st);
cudaError_t launch_mma_one(const MmaParams& p, int64_t groups, Carve& ws, cudaStream_t st);
cudaError_t launch_mma_two(const MmaParams& p, int64_t groups, Carve& ws, cudaStream_t st);

}  // namespace q8
