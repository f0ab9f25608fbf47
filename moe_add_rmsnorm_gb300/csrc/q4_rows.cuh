// Products of 4-bit weights with several activation rows: the projection, and a chunk's experts (each expert's weights with
// the rows that chose it: gate-up with SwiGLU, and down-and-combine).
//
// A first launch lays the activation rows out as f16 parts (q4.cuh) in the order of the products' operands; a second one
// multiplies.  There a warp takes two tiles of 16 weight rows (gate-up: 16 gate rows and the 16 up rows beside them) by up
// to two tiles of eight columns, a column being one part of one activation row.  Weights and activation parts come through
// rings of asynchronous 16-byte copies: the weights' is the warp's own, from where one matrix load gives each lane the words
// it multiplies; the activation's is the CTA's, whose warps read the same columns.  A block's dots are scaled, two sums an
// instruction, by the weights' scale (and a quantized activation's; an f32 row has one unit, taken out at the end).
// What bounds it is instructions: a warp's chunk of 32 rows by 128 values is some 440 of them, of which unpacking, needed once
// however few the columns, is the larger part; 16 warps an SM issue in 56% of the cycles.  Measured, replayed: 24 rows by 8 of
// 128 experts of 2048 x 768, one-word activations, 93 us (250 MB; 36.6 at the measured copy rate), 8 f32 rows by 8192 x 4096
// 12.1.  The columns' ring is the CTA's since operands from L1 cost their latency every chunk (197 -> 131 us).
#pragma once
#include "ffn4.h"
#include "q4.cuh"

namespace q8 {

constexpr int kWarps = 8;    // a CTA
constexpr int kStages = 4;   // of the rings: a stage is a chunk of four blocks for each of the warps that share a tile
constexpr int kRowCtas = 2;  // an SM's CTAs (three leave a lane 80 registers, which spill: a batch's experts 98 -> 164 us)
constexpr int NT = 2;        // tiles of eight columns a pass (four: 60 rows by 6 of 64 experts, 2048 x 1408, 148 -> 201 us)
constexpr int kTileBytes = 2 * 16 * 64;

struct RowsParams {
    Q4View w0, w1;
    Q4Act act;
    int kind;
    int64_t E, out_rows;
    int R, K;            // activation rows of the call and choices a row
    int64_t act_rows;    // rows that are laid out
    PlanPtrs plan;
    const int32_t* ids;
    uint4* parts;        // [act_rows][4 * chunks][parts][4]
    float* scales;       // f32: [act_rows], a row's unit; else [act_rows][4 * chunks] (two words: each twice)
    float* y;
    int64_t y_stride;
    float* out;          // down: [R * K][out_rows]
    int chunks, wk, row_tiles;
};

// A CTA lays one activation row out at a time.
template <int FORM>
__global__ void __launch_bounds__(256) q4_parts_kernel(const RowsParams p) {
    constexpr int PARTS = FORM == FORM_ONE ? 1 : 2;
    __shared__ float most[2][8];
    griddep_wait();    // the launch before has ended, which the products' launch takes for granted from its start on
    griddep_launch();
    const int octets = 16 * p.chunks, cols = p.w0.cols, lane = threadIdx.x & 31;
    int buf = 0;
    for (int64_t r = blockIdx.x; r < p.act_rows; r += gridDim.x, buf ^= 1) {
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
            for (int i = 0; i < 8; ++i) m = fmaxf(m, most[buf][i]);
        }
        for (int o = threadIdx.x; o < octets; o += blockDim.x) {
            ActParts a;
            if (FORM == FORM_F32) {
                float x[8];
                act_values(p.act, r, o, cols, x);
                a = split_values(x, m);
                if (o == 0) p.scales[r] = a.scale;
            } else {
                a = act_words(p.act, r, o, cols);
                const int64_t b = r * (octets / 4) + (o >> 2);
                if ((o & 3) == 0) {
                    if (FORM == FORM_ONE) p.scales[b] = a.scale;
                    else reinterpret_cast<float2*>(p.scales)[b] = make_float2(a.scale, a.scale);
                }
            }
            uint4* at = p.parts + (r * octets + (o & ~3)) * PARTS + (o & 3);
            at[0] = a.hi;
            if (PARTS == 2) at[4] = a.lo;
        }
    }
}

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void zero16(uint32_t dst) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(dst), "r"(0) : "memory");
}
template <int N>
__device__ __forceinline__ void copy_small(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(N) : "memory");
}

__device__ __forceinline__ void load_matrices(uint32_t (&m)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(m[0]), "=r"(m[1]), "=r"(m[2]), "=r"(m[3]) : "r"(at) : "memory");
}

// d = a b, without an addend.
__device__ __forceinline__ void mma16_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                            uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
                 : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// A warp's chunk: the four blocks of its 32 rows (matrix tiles from `mat` on) by the first TN tiles of columns (at `bs`).  Without a
// branch for every tile of columns, so that the products of one hide the scaling of another.  so, zo: the scales and zero
// points of the chunk's groups in row g + 8 (t & 1) of tile t >> 1; 2^same blocks share one.
template <int FORM, int TN>
__device__ __forceinline__ void multiply_chunk(uint32_t mat, const char* bs, const float (&so)[4], const uint32_t (&zo)[4],
                                               bool has_z, int same, float2 (&acc)[2][NT][2]) {
    constexpr int BCHUNK = NT * 8 * 4 * 64;
    const int lane = threadIdx.x & 31, quad = lane & ~3;
    const uint4* bcol = reinterpret_cast<const uint4*>(bs) + lane;
    const float2* bscale = reinterpret_cast<const float2*>(bs + BCHUNK) + (lane & 3);
    float sw[2][2];
    uint32_t zc[2][2], zf[2][2];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int i = 0; i < 2; ++i) zero_forms(8, zc[m][i], zf[m][i]);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        uint32_t words[2][4];  // [m][block 2 half: rows g, rows g + 8; block 2 half + 1: the same]
#pragma unroll
        for (int m = 0; m < 2; ++m) load_matrices(words[m], (mat + m * 1024) ^ (32 * half));
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int b = 2 * half + k;
            if ((b & ((1 << same) - 1)) == 0) {  // a group starts: its number in the chunk is b >> same
                const float sg = b == 2 && same ? so[1] : so[b];
                const uint32_t zg = b == 2 && same ? zo[1] : zo[b];
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        sw[m][i] = __shfl_sync(0xffffffffu, sg, quad + 2 * m + i);
                        if (has_z) {
                            zc[m][i] = __shfl_sync(0xffffffffu, zg, quad + 2 * m + i);
                            zf[m][i] = zero_less(zc[m][i]);
                        }
                    }
            }
            uint32_t h[2][2][4];
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int i = 0; i < 2; ++i) words_f16(words[m][2 * k + i], zc[m][i], zf[m][i], h[m][i]);
#pragma unroll
            for (int n = 0; n < TN; ++n) {
                const uint4 x = bcol[(b * NT + n) * 32];
                float2 sx = make_float2(1.f, 1.f);
                if (FORM != FORM_F32) sx = bscale[(b * NT + n) * 4];
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    float d[4];
                    mma16_first(d, h[m][0][0], h[m][1][0], h[m][0][1], h[m][1][1], x.x, x.y);
                    mma16(d, h[m][0][2], h[m][1][2], h[m][0][3], h[m][1][3], x.z, x.w);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float2 w = make_float2(sw[m][i], sw[m][i]);
                        pair_fma(acc[m][n][i], FORM == FORM_F32 ? w : pair_mul(w, sx), d[2 * i], d[2 * i + 1]);
                    }
                }
            }
        }
    }
}

template <int FORM>
__global__ void __launch_bounds__(32 * kWarps, kRowCtas) q4_rows_kernel(const RowsParams p) {
    constexpr int PARTS = FORM == FORM_ONE ? 1 : 2;
    constexpr int COLS = 8 / PARTS;  // activation rows a tile of columns
    constexpr int NC = NT * COLS;
    constexpr int BCHUNK = NT * 8 * 4 * 64;                          // a chunk's columns: [block][column][4 x 16 bytes]
    constexpr int SCHUNK = FORM == FORM_F32 ? 0 : 4 * NT * 8 * 4;    // and scales: [block][column] (two words: a row's twice)
    extern __shared__ __align__(128) char smem[];
    __shared__ int cols[NC];           // the choices (dense: activation rows) of the columns, -1: none
    __shared__ uint32_t rowat[NC];     // their activation rows
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int side = kWarps / p.wk, tile = blockIdx.x * side + w / p.wk, part_of = w % p.wk;
    const int nb = p.w0.cols >> 5, ngroups = p.w0.cols >> p.w0.group_log2, row_bytes = p.w0.cols >> 1;
    const int steps = (p.chunks + p.wk - 1) / p.wk;
    // The rings.  Of a chunk of weights, block t of row r of 16 stands at 64 r + 16 (t ^ (r >> 1 & 3)), so that the eight rows
    // of a matrix load lie in different banks.
    char* columns = smem + kWarps * kStages * kTileBytes;
    const uint32_t base_a = (uint32_t)__cvta_generic_to_shared(smem) + w * (kStages * kTileBytes);
    const uint32_t base_b = (uint32_t)__cvta_generic_to_shared(columns), stage_b = p.wk * (BCHUNK + SCHUNK);
    const uint32_t ring_at = base_a + g * 64 + ((t ^ ((g >> 1) & 3)) << 4);
    const uint32_t matrix_at = base_a + (lane & 15) * 64 + (((lane >> 4) ^ ((lane >> 1) & 3)) << 4);
    // Of a chunk of columns the thread copies unit (block, part, word) of rows unit_row, + 2 kWarps / PARTS, ...
    constexpr int NU = NT * 8 * 16 / (32 * kWarps);
    const int unit_of = threadIdx.x % (16 * PARTS), unit_row = threadIdx.x / (16 * PARTS);
    const uint32_t unit_at = (((unit_of / (4 * PARTS)) * NT * 8 + unit_row * PARTS + (unit_of >> 2) % PARTS) * 4 + (unit_of & 3)) * 16;
    const uint32_t scale_at = BCHUNK + ((threadIdx.x % 4) * NT * 8 + threadIdx.x / 4 * PARTS) * 4;
    const bool has_z = p.w0.z != nullptr;
    const int same = p.w0.group_log2 - 5, per_chunk = 4 >> same;
    const int total = p.R * p.K;
    const bool gate_up = p.kind == Q4_GATE_UP;
    const Q4View& second = gate_up ? p.w1 : p.w0;
    // a chunk's scales (and zero points) in one load, where every row's stand at a multiple of their size
    const bool wide = ngroups % per_chunk == 0 && (((uintptr_t)p.w0.s | (uintptr_t)second.s) % (2 * per_chunk)) == 0 &&
                      (((uintptr_t)p.w0.z | (uintptr_t)second.z) % per_chunk) == 0;
    bool ready = false;
    int groups = 1;
    if (p.kind != Q4_DENSE) groups = p.plan.active ? min(max(p.plan.active[0], 0), (int)min(p.E, (int64_t)total)) : p.K;
    griddep_launch();
    for (int a = blockIdx.y; a < groups; a += gridDim.y) {
        int e = 0, first = 0, count = p.R;
        if (p.kind != Q4_DENSE) {
            e = p.plan.active ? p.plan.active[1 + a] : p.ids[a];  // (one row has no plan: every choice is a group)
            if (e < 0 || e >= p.E) continue;
            first = p.plan.active ? max(p.plan.offsets[e], 0) : a;
            count = p.plan.active ? min(p.plan.offsets[e + 1], total) - first : 1;
        }
        // The lane's rows of the two weight tiles, rows g and g + 8 of each (they clamp to the group's last row), as offsets
        // from the first tile row's words and scales, which run on from chunk to chunk.
        const int64_t base = (int64_t)e * p.out_rows;
        const int r0 = (gate_up ? 16 : 32) * tile, last = (int)p.out_rows - 1, top = min(r0, last);
        const uint8_t *qa = p.w0.q + (base + top) * row_bytes, *qb = second.q + (base + top) * row_bytes;
        int woff[2][2];
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int row = min(r0 + (gate_up ? 0 : 16 * m) + g + 8 * i, last) - top;
                woff[m][i] = row * row_bytes + 16 * t;
            }
        // Of scales a lane loads those of one of its four rows.
        const int64_t srow = (base + min(r0 + (gate_up ? 0 : 16 * (t >> 1)) + g + 8 * (t & 1), last)) * ngroups;
        const uint16_t* sp = (t >> 1 ? second.s : p.w0.s) + srow;
        const uint8_t* zp = (t >> 1 ? second.z : p.w0.z) + srow;
        for (int ct = blockIdx.z; ct * NC < count; ct += gridDim.z) {
            const int tiles = min((count - ct * NC + COLS - 1) / COLS, NT);
            uint2 s;         // the next chunk's scales and zero points, packed
            uint32_t z;
            int sc = part_of;  // that chunk
            auto scales = [&]() {
                s = make_uint2(0, 0), z = 0;
                if (sc < p.chunks) {
                    const int at = sc * per_chunk;
                    if (!wide) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            if (j >= per_chunk || at + j >= ngroups) break;
                            (j < 2 ? s.x : s.y) |= (uint32_t)__ldg(sp + at + j) << (16 * (j & 1));
                            if (has_z) z |= (uint32_t)__ldg(zp + at + j) << (8 * j);
                        }
                    } else if (per_chunk == 4) {
                        s = __ldg(reinterpret_cast<const uint2*>(sp + at));
                        if (has_z) z = __ldg(reinterpret_cast<const uint32_t*>(zp + at));
                    } else if (per_chunk == 2) {
                        s.x = __ldg(reinterpret_cast<const uint32_t*>(sp + at));
                        if (has_z) z = __ldg(reinterpret_cast<const uint16_t*>(zp + at));
                    } else {
                        s.x = __ldg(sp + at);
                        if (has_z) z = __ldg(zp + at);
                    }
                }
                sc += p.wk;
            };
            int wc = part_of;  // the chunk of weights that is fetched next, its place in the ring, and of the columns'
            uint32_t wat = 0, bat = 0;
            int bc = 0;
            auto fetch_weights = [&]() {
                if (wc < p.chunks) {
                    const uint32_t to = ring_at + wat;
                    const int from = 64 * wc;
                    if (4 * wc + t < nb) {
#pragma unroll
                        for (int m = 0; m < 2; ++m)
#pragma unroll
                            for (int i = 0; i < 2; ++i)
                                copy16(to + m * 1024 + i * 512, (m == 0 ? qa : qb) + (woff[m][i] + from));
                    } else {  // (columns past the last: zeros in the activations, anything finite here)
#pragma unroll
                        for (int m = 0; m < 4; ++m) zero16(to + m * 512);
                    }
                }
                wc += p.wk;
                wat = wat == (kStages - 1) * kTileBytes ? 0 : wat + kTileBytes;
            };
            uint32_t goff[NU];  // the thread's 16-byte units of a chunk of the columns
            const float* sfrom = p.scales;  // and its scale (words: of block threadIdx.x % 4 of row threadIdx.x / 4)
            const int rows_here = tiles * COLS;
            auto fetch_columns = [&]() {  // all warps: the stage's chunks of the columns
                for (int j = 0; j < p.wk && bc < p.chunks; ++j, ++bc) {
                    const uint32_t to = base_b + bat + j * (BCHUNK + SCHUNK) + unit_at;
#pragma unroll
                    for (int k = 0; k < NU; ++k)
                        if (unit_row + k * (kWarps * 2 / PARTS) < rows_here)
                            copy16(to + k * 1024, p.parts + (goff[k] + (uint32_t)bc * (16 * PARTS)));
                    if (FORM != FORM_F32 && (int)threadIdx.x < 4 * rows_here) {
                        const uint32_t sto = base_b + bat + j * (BCHUNK + SCHUNK) + scale_at;
                        if (FORM == FORM_ONE) copy_small<4>(sto, sfrom + 4 * bc);
                        else copy_small<8>(sto, sfrom + 8 * bc);
                    }
                }
                bat = bat == (kStages - 1) * stage_b ? 0 : bat + stage_b;
            };
            // weights first: they depend on no launch before
            scales();
            fetch_weights();
            __syncthreads();  // (the columns before these have been used)
            if (threadIdx.x < NC) {
                const int i = ct * NC + threadIdx.x;
                int c = i < count ? (p.kind == Q4_DENSE ? i : p.plan.active ? p.plan.lists[first + i] : first) : -1;
                if (c < 0 || c >= total) c = -1;
                cols[threadIdx.x] = c;
                rowat[threadIdx.x] = gate_up ? max(c, 0) / p.K : max(c, 0);
            }
            __syncthreads();
#pragma unroll
            for (int k = 0; k < NU; ++k)
                goff[k] = rowat[min(unit_row + k * (kWarps * 2 / PARTS), NC - 1)] * (uint32_t)(16 * PARTS * p.chunks) + unit_of;
            if (FORM != FORM_F32)
                sfrom = p.scales + ((size_t)rowat[min((int)threadIdx.x / 4, NC - 1)] * (4 * p.chunks) + threadIdx.x % 4) * PARTS;
            if (!ready) griddep_wait(), ready = true;  // the activation parts
            fetch_columns();
            asm volatile("cp.async.commit_group;" ::: "memory");
#pragma unroll
            for (int i = 1; i < kStages - 1; ++i) {
                fetch_weights();
                fetch_columns();
                asm volatile("cp.async.commit_group;" ::: "memory");
            }
            float2 acc[2][NT][2] = {};  // [tile][columns][row g, g + 8]: columns 2 t and 2 t + 1
            uint32_t at = 0, bt = 0;
            for (int c = part_of, step = 0; step < steps; ++step, c += p.wk) {
                asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
                __syncthreads();
                fetch_weights();
                fetch_columns();
                asm volatile("cp.async.commit_group;" ::: "memory");
                float so[4];
                uint32_t zo[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    so[j] = scale_f32(((j < 2 ? s.x : s.y) >> (16 * (j & 1))) & 0xffffu, p.w0.bf16);
                    zo[j] = 0x64006400u | (((z >> (8 * j)) & 0xffu) * 0x10001u);
                }
                scales();
                if (c < p.chunks) {
                    const uint32_t mat = matrix_at + at;
                    const char* bs = columns + bt + part_of * (BCHUNK + SCHUNK);
                    if (tiles > 1) multiply_chunk<FORM, 2>(mat, bs, so, zo, has_z, same, acc);
                    else multiply_chunk<FORM, 1>(mat, bs, so, zo, has_z, same, acc);
                }
                at = at == (kStages - 1) * kTileBytes ? 0 : at + kTileBytes;
                bt = bt == (kStages - 1) * stage_b ? 0 : bt + stage_b;
            }
            asm volatile("cp.async.wait_group 0;" ::: "memory");
            if (p.wk > 1) {  // the warps' sums of the tile, in the order of their parts
                __syncthreads();
                float2* red = reinterpret_cast<float2*>(smem);
                if (part_of) {
#pragma unroll
                    for (int m = 0; m < 2; ++m)
#pragma unroll
                        for (int n = 0; n < NT; ++n)
#pragma unroll
                            for (int i = 0; i < 2; ++i) red[(w * 4 * NT + (m * NT + n) * 2 + i) * 32 + lane] = acc[m][n][i];
                }
                __syncthreads();
                if (part_of == 0) {
                    for (int k = 1; k < p.wk; ++k)
#pragma unroll
                        for (int m = 0; m < 2; ++m)
#pragma unroll
                            for (int n = 0; n < NT; ++n)
#pragma unroll
                                for (int i = 0; i < 2; ++i) {
                                    const float2 v = red[((w + k) * 4 * NT + (m * NT + n) * 2 + i) * 32 + lane];
                                    acc[m][n][i].x += v.x, acc[m][n][i].y += v.y;
                                }
                }
            }
            if (part_of == 0 && tile < p.row_tiles) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int j = 0; j < 2 / PARTS; ++j) {
                            const int at = n * COLS + (2 / PARTS) * t + j, c = cols[at];
                            if (n >= tiles || c < 0) continue;
                            float v[2];
#pragma unroll
                            for (int m = 0; m < 2; ++m) {
                                v[m] = PARTS == 2 ? acc[m][n][i].x + acc[m][n][i].y : j ? acc[m][n][i].y : acc[m][n][i].x;
                                if (FORM == FORM_F32) v[m] *= p.scales[rowat[at]];
                            }
                            const int r = r0 + g + 8 * i;
                            if (gate_up) {
                                if (r <= last) p.y[c * p.y_stride + r] = silu_f32(v[0]) * v[1];
                            } else {
                                float* to = p.kind == Q4_DENSE ? p.y + c * p.y_stride : p.out + c * p.out_rows;
                                if (r <= last) to[r] = v[0];
                                if (r + 16 <= last) to[r + 16] = v[1];
                            }
                        }
            }
            __syncthreads();  // (the rings take the next columns)
        }
    }
    if (!ready) griddep_wait();  // (a grid ends after the launch before it, whatever its CTAs had to do)
}

constexpr size_t kRowsSmem = 220 << 10;

template <int FORM>
cudaError_t run_rows(RowsParams p, int64_t groups, cudaStream_t st) {
    constexpr int NC = NT * 8 / (FORM == FORM_ONE ? 1 : 2);
    const int sms = device_info().sms;
    auto smem = [&](int wk) {
        return (size_t)kStages * (kWarps * kTileBytes + wk * (NT * 2048 + (FORM == FORM_F32 ? 0 : NT * 128)));
    };
    const int64_t zs = p.kind == Q4_DENSE ? min((int64_t)(p.R + NC - 1) / NC, (int64_t)65535) : 1;
    // Warps that share a tile: those with the fewest steps in all, waves of CTAs times a CTA's steps and three for its ends.
    // Measured, us, 1, 2, 4 and 8 warps: 8 rows by 8192 x 4096 33, 19, 12 and 15; by 2048 x 2048 17.5, 10.8, 7.3 and 5.6.
    int64_t fewest = INT64_MAX;
    for (int wk = 1; wk <= kWarps && wk <= p.chunks && smem(wk) <= kRowsSmem; wk *= 2) {
        const int64_t ctas = (p.row_tiles + kWarps / wk - 1) / (kWarps / wk) * groups * zs;
        const int64_t at_once = sms * min((int64_t)(kRowsSmem / smem(wk)), (int64_t)kRowCtas);
        const int64_t steps = (ctas + at_once - 1) / at_once * ((p.chunks + wk - 1) / wk + 3);
        if (steps < fewest) fewest = steps, p.wk = wk;
    }
    const int side = kWarps / p.wk;
    const dim3 grid((unsigned)((p.row_tiles + side - 1) / side), (unsigned)min(groups, (int64_t)65535), (unsigned)zs);
    static std::atomic<uint64_t> done;
    const cudaError_t e = allow_smem(q4_rows_kernel<FORM>, kRowsSmem, done);
    if (e != cudaSuccess) return e;
    return launch(q4_rows_kernel<FORM>, grid, dim3(32 * kWarps), smem(p.wk), st, 1, p);
}

// Both launches of a call of at most `groups` groups of rows.
template <int FORM>
cudaError_t launch_rows(const RowsParams& p, int64_t groups, cudaStream_t st) {
    const dim3 lay((unsigned)min(p.act_rows, (int64_t)device_info().sms * 8));
    const cudaError_t e = launch(q4_parts_kernel<FORM>, lay, dim3(256), 0, st, 1, p);
    if (e != cudaSuccess) return e;
    return run_rows<FORM>(p, groups, st);
}

// One file each, so that they compile beside one another.
cudaError_t launch_rows_f32(const RowsParams& p, int64_t groups, cudaStream_t st);
cudaError_t launch_rows_one(const RowsParams& p, int64_t groups, cudaStream_t st);
cudaError_t launch_rows_two(const RowsParams& p, int64_t groups, cudaStream_t st);

}  // namespace q8
