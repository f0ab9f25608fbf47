// Products of 4-bit weights with one activation row: the projection, and a row's experts (gate-up with SwiGLU, and
// down-and-combine).
//
// The work is bound by the weights' bytes, which lanes read straight into registers, 16 bytes (a whole 32-value block of one
// row) a load.  A warp takes 16 rows by chunks of four blocks: lane (g, t) holds block t of rows g and g + 8, which
// is an A operand of the warp-wide f16 product if the product's sum over t is kept apart.  Its eight columns do that: column
// (j, p) holds part p of the activation's block j, and zeros where the lanes with t != j read.  Lane (g, t) then receives the
// two parts' dots of its own block of its own rows, and scales them by the scales it loaded.  So no weight passes through
// shared memory or a shuffle, and every group size costs the same.
#include "ffn4.h"
#include "q4.cuh"

namespace q8 {
namespace {

constexpr int kRowWarps = 8;
constexpr int kBlockBytes = 144;  // a block's two parts of 64 bytes, 16 more so that four blocks lie in different banks

struct RowParams {
    Q4View w0, w1;
    Q4Act act;
    int64_t E, out_rows;  // rows a group
    int K;
    const int32_t* ids;
    const float *gates, *residual;
    float* y;
    int chunks;      // of four blocks, a row
    int wk;          // warps that share a tile's columns
    int tiles;       // of 16 * MT rows (all groups')
    int row_tiles;   // a group's
    int batch;       // down: hidden rows in shared memory at a time
    int slices;      // down: warps' tasks a hidden row
    uint32_t vec;    // bytes of a row's parts in shared memory
};

// The four-block chunk `c` of rows r and r + 8 (while below `rows`) of w.
struct Chunk {
    uint4 w[2];
    uint32_t s[2], z[2];
};

__device__ __forceinline__ void fetch(Chunk& q, const Q4View& w, int64_t row0, int r, int64_t rows, int c, int nb) {
    const int t = threadIdx.x & 3, b = 4 * c + t;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        if (r + 8 * i < rows && b < nb) {
            const int64_t row = row0 + r + 8 * i;
            const uint8_t* p = w.q + row * (w.cols >> 1) + 16 * b;
            asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                         : "=r"(q.w[i].x), "=r"(q.w[i].y), "=r"(q.w[i].z), "=r"(q.w[i].w)
                         : "l"(p));
            const int64_t g = row * (w.cols >> w.group_log2) + ((32 * b) >> w.group_log2);
            q.s[i] = __ldg(w.s + g);
            q.z[i] = w.z ? __ldg(w.z + g) : 8u;
        } else {
            q.w[i] = make_uint4(0, 0, 0, 0);
            q.s[i] = 0u;
            q.z[i] = 8u;
        }
    }
}

// acc[i] += the chunk's block t of row g + 8 i times the activation's.
__device__ __forceinline__ void multiply(const Chunk& q, const uint4 (&b)[4], float sx, int bf16, float (&acc)[2]) {
    float d[4] = {0.f, 0.f, 0.f, 0.f};
    uint32_t zc[2], zf[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) zero_forms(q.z[i], zc[i], zf[i]);
#pragma unroll
    for (int m = 0; m < 4; ++m) {
        const uint32_t w0 = m == 0 ? q.w[0].x : m == 1 ? q.w[0].y : m == 2 ? q.w[0].z : q.w[0].w;
        const uint32_t w1 = m == 0 ? q.w[1].x : m == 1 ? q.w[1].y : m == 2 ? q.w[1].z : q.w[1].w;
        uint32_t h0[4], h1[4];
        words_f16(w0, zc[0], zf[0], h0);
        words_f16(w1, zc[1], zf[1], h1);
        mma16(d, h0[0], h1[0], h0[1], h1[1], b[m].x, b[m].y);
        mma16(d, h0[2], h1[2], h0[3], h1[3], b[m].z, b[m].w);
    }
    acc[0] = fmaf(scale_f32(q.s[0], bf16) * sx, d[0] + d[1], acc[0]);
    acc[1] = fmaf(scale_f32(q.s[1], bf16) * sx, d[2] + d[3], acc[1]);
}

// Rows first .. first + n of the activation as parts in shared memory.
__device__ __forceinline__ void stage_rows(const RowParams& p, char* vecs, int first, int n) {
    const int octets = 4 * 4 * p.chunks, cols = p.w0.cols;  // eight values each, up to whole chunks
    for (int i = threadIdx.x; i < ((n * octets + 31) & ~31); i += blockDim.x) {  // whole warps: quads share a block
        const int v = i / octets, o = i - v * octets, b = o >> 2;
        ActParts a;
        if (p.act.x) {  // a block's four lanes share its unit
            float x[8];
            act_values(p.act, first + min(v, n - 1), v < n ? o : octets, cols, x);
            float m = finite_max(x);
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
            a = split_values(x, m);
        } else {
            a = act_words(p.act, first + min(v, n - 1), o, cols);
        }
        if (v >= n) continue;
        char* at = vecs + v * p.vec + b * kBlockBytes + (o & 3) * 16;
        *reinterpret_cast<uint4*>(at) = a.hi;
        *reinterpret_cast<uint4*>(at + 64) = a.lo;
        if ((o & 3) == 0) *reinterpret_cast<float*>(vecs + v * p.vec + 4 * p.chunks * kBlockBytes + 4 * b) = a.scale;
    }
}

// A lane's operand of the product: part g & 1 of block t for the lanes that hold a column of their own block, else zeros.
struct Operand {
    const char *at, *scale;
    uint32_t step;
};
__device__ __forceinline__ Operand operand(const RowParams& p, const char* vec, const char* zeros) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const bool own = (g >> 1) == t;
    return Operand{own ? vec + t * kBlockBytes + (g & 1) * 64 : zeros, vec + 4 * p.chunks * kBlockBytes + 4 * t,
                   own ? 4u * kBlockBytes : 0u};
}
__device__ __forceinline__ void load_operand(const Operand& o, int c, uint4 (&b)[4], float& sx) {
#pragma unroll
    for (int m = 0; m < 4; ++m) b[m] = *reinterpret_cast<const uint4*>(o.at + c * o.step + 16 * m);
    sx = *reinterpret_cast<const float*>(o.scale + 16 * c);
}

__device__ __forceinline__ float quad_sum(float v) {
    v += __shfl_xor_sync(0xffffffffu, v, 1);
    return v + __shfl_xor_sync(0xffffffffu, v, 2);
}

// The projection (MT = 1: a tile is 16 rows) and the gate-up (MT = 2: a tile is 16 gate rows and the up rows beside them).
// wk warps share a tile, each `mine` chunks of its columns; a warp's chunks follow one another over all its tiles, DEPTH of
// them on their way.
template <int MT, int DEPTH>
__global__ void __launch_bounds__(32 * kRowWarps, 2) q4_row_kernel(const RowParams p) {
    extern __shared__ __align__(16) char smem[];
    __shared__ float part[2][kRowWarps][MT][16];
    __shared__ uint4 zeros[4];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int nb = p.w0.cols >> 5, side = kRowWarps / p.wk;  // tiles that the CTA's warps take side by side
    const int mine = (p.chunks + p.wk - 1) / p.wk, c0 = (w % p.wk) * mine;
    const int stride = gridDim.x * side, first = blockIdx.x * side + w / p.wk;
    const int rounds = (p.tiles - (int)blockIdx.x * side + stride - 1) / stride;  // the CTA's, alike in all its warps
    // the chunk that is fetched next: its tile, place, group's first row and rows
    int tile = first, at = 0, r0 = 0;
    int64_t base = 0, rows = 0;
    auto locate = [&]() {
        rows = 0;
        if (tile >= p.tiles) return;
        const int group = tile / p.row_tiles, e = p.ids ? p.ids[group] : 0;
        r0 = 16 * (tile - group * p.row_tiles);
        if (e >= 0 && e < p.E) base = e * p.out_rows, rows = p.out_rows;
    };
    Chunk q[DEPTH][MT];
    auto next = [&](Chunk (&c)[MT]) {
        fetch(c[0], p.w0, base, r0 + g, rows, c0 + at, nb);
        if (MT == 2) fetch(c[MT - 1], p.w1, base, r0 + g, rows, c0 + at, nb);
        if (++at == mine) {
            at = 0;
            tile += stride;
            locate();
        }
    };
    locate();
#pragma unroll
    for (int i = 0; i < DEPTH; ++i) next(q[i]);
    if (threadIdx.x < 4) zeros[threadIdx.x] = make_uint4(0, 0, 0, 0);
    stage_rows(p, smem, 0, 1);
    __syncthreads();
    const Operand o = operand(p, smem, reinterpret_cast<const char*>(zeros));
    float acc[MT][2] = {};
    int done = 0, own = first, buf = 0;
    const int total = rounds * mine;
    for (int it = 0; it < total; it += DEPTH) {
#pragma unroll
        for (int k = 0; k < DEPTH; ++k) {
            if (it + k >= total) break;
            if (c0 + done < p.chunks) {
                uint4 b[4];
                float sx;
                load_operand(o, c0 + done, b, sx);
#pragma unroll
                for (int m = 0; m < MT; ++m) multiply(q[k][m], b, sx, p.w0.bf16, acc[m]);
            }
            next(q[k]);
            if (++done < mine) continue;
            // the tile's end: the warps' sums in the order of their columns
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float v = quad_sum(acc[m][i]);
                    if (t == 0) part[buf][w][m][g + 8 * i] = v;
                    acc[m][i] = 0.f;
                }
            if (p.wk > 1) __syncthreads();
            else __syncwarp();
            if (w % p.wk == 0 && lane < 16 && own < p.tiles) {
                const int group = own / p.row_tiles, r = 16 * (own - group * p.row_tiles) + lane;
                float v[MT] = {};
                for (int j = 0; j < p.wk; ++j)
#pragma unroll
                    for (int m = 0; m < MT; ++m) v[m] += part[buf][w + j][m][lane];
                bool ok = r < p.out_rows;
                if (p.ids && ok) {
                    const int e = p.ids[group];
                    ok = e >= 0 && e < p.E;
                }
                if (ok) p.y[group * p.out_rows + r] = MT == 2 ? silu_f32(v[0]) * v[MT - 1] : v[0];
            }
            buf ^= 1;  // (the next tile's sums go to the other half: one barrier a tile)
            done = 0;
            own += stride;
        }
    }
}

// Down-and-combine: a CTA takes 16 output rows of all the row's experts, its warps (hidden row, part of its columns) tasks;
// the sums meet in shared memory and are added up in the order of the experts.  Hidden rows come `batch` at a time.
template <int DEPTH>
__global__ void __launch_bounds__(32 * kRowWarps, 2) q4_down_row_kernel(const RowParams p) {
    extern __shared__ __align__(16) char smem[];
    __shared__ uint4 zeros[4];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int nb = p.w0.cols >> 5, r0 = 16 * blockIdx.x;
    float* part = reinterpret_cast<float*>(smem + (size_t)p.batch * p.vec);  // [K * slices][16]
    const int mine = (p.chunks + p.slices - 1) / p.slices;
    const int per = (p.batch * p.slices + kRowWarps - 1) / kRowWarps;  // tasks a warp and batch
    const int batches = (p.K + p.batch - 1) / p.batch;
    // the chunk that is fetched next
    int task = 0, batch = 0, at = 0, c0 = 0;
    int64_t base = 0, rows = 0;
    auto expert = [&](int j) {  // the hidden row's expert, or -1
        const int e = j < p.K ? p.ids[j] : -1;
        return e >= 0 && e < p.E ? e : -1;
    };
    auto place = [&](int b, int i, int& j, int& s) {  // task i of this warp in batch b: hidden row and part (j = K: none)
        const int k = i * kRowWarps + w;
        s = k % p.slices;
        j = k / p.slices < p.batch && b < batches ? b * p.batch + k / p.slices : p.K;
        j = min(j, p.K);
    };
    auto locate = [&]() {
        int j, s;
        place(batch, task, j, s);
        const int e = expert(j);
        c0 = s * mine;
        rows = 0;
        if (e >= 0) base = e * p.out_rows, rows = p.out_rows;
    };
    Chunk q[DEPTH];
    auto next = [&](Chunk& c) {
        fetch(c, p.w0, base, r0 + g, at < mine ? rows : 0, c0 + at, nb);
        if (++at == mine) {
            at = 0;
            if (++task == per) task = 0, ++batch;
            locate();
        }
    };
    locate();
#pragma unroll
    for (int i = 0; i < DEPTH; ++i) next(q[i]);
    if (threadIdx.x < 4) zeros[threadIdx.x] = make_uint4(0, 0, 0, 0);
    float acc[2] = {};
    int done = 0, my_task = 0, my_batch = 0, j, s;
    Operand o = {};
    const int total = batches * per * mine;
    for (int it = 0; it < total; it += DEPTH) {
#pragma unroll
        for (int k = 0; k < DEPTH; ++k) {
            if (it + k >= total) break;
            if (done == 0) {
                if (my_task == 0) {  // (all warps alike)
                    if (my_batch > 0) __syncthreads();
                    stage_rows(p, smem, my_batch * p.batch, min(p.batch, p.K - my_batch * p.batch));
                    __syncthreads();
                }
                place(my_batch, my_task, j, s);
                o = operand(p, smem + (size_t)(min(j, p.K - 1) - my_batch * p.batch) * p.vec, reinterpret_cast<const char*>(zeros));
            }
            if (j < p.K && s * mine + done < p.chunks) {
                uint4 b[4];
                float sx;
                load_operand(o, s * mine + done, b, sx);
                multiply(q[k], b, sx, p.w0.bf16, acc);
            }
            next(q[k]);
            if (++done < mine) continue;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float v = quad_sum(acc[i]);
                if (t == 0 && j < p.K) part[(j * p.slices + s) * 16 + g + 8 * i] = v;
                acc[i] = 0.f;
            }
            done = 0;
            if (++my_task == per) my_task = 0, ++my_batch;
        }
    }
    __syncthreads();
    const int r = r0 + threadIdx.x;
    if (threadIdx.x >= 16 || r >= p.out_rows) return;
    float sum = 0.f;
    for (int k = 0; k < p.K; ++k) {
        if (expert(k) < 0) continue;
        float v = 0.f;
        for (int i = 0; i < p.slices; ++i) v += part[(k * p.slices + i) * 16 + threadIdx.x];
        sum = fmaf(p.gates[k], v, sum);
    }
    p.y[r] = p.residual ? p.residual[r] + sum : sum;
}

constexpr size_t kRowSmem = 200 << 10;

template <typename Kern>
cudaError_t allow_smem(Kern kernel, size_t smem) {
    return smem > (48 << 10) - 4096 ? cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem)
                                    : cudaSuccess;
}

}  // namespace

cudaError_t launch_q4_row(const Q4Call& c, cudaStream_t st) {
    RowParams p = {};
    p.w0 = c.w0;
    p.w1 = c.w1;
    p.act = c.act;
    p.E = c.E;
    p.out_rows = c.out_rows;
    p.K = c.K;
    p.ids = c.kind == Q4_DENSE ? nullptr : c.ids;
    p.gates = c.gates;
    p.residual = c.residual;
    p.y = c.y;
    p.chunks = (c.w0.cols + 127) / 128;
    p.vec = (uint32_t)p.chunks * (4 * kBlockBytes + 16);
    p.row_tiles = (int)((c.out_rows + 15) / 16);
    const int sms = device_info().sms;
    if (c.kind == Q4_DOWN) {
        p.batch = (int)min((size_t)c.K, kRowSmem / p.vec);
        // parts of a hidden row: what leaves the warps the fewest chunks one after another
        p.slices = 1;
        auto steps = [&](int s) { return (p.batch * s + kRowWarps - 1) / kRowWarps * ((p.chunks + s - 1) / s); };
        for (int s = 2; s <= 8 && s <= p.chunks; ++s)
            if (steps(s) < steps(p.slices)) p.slices = s;
        const size_t smem = (size_t)p.batch * p.vec + (size_t)c.K * p.slices * 64;
        const cudaError_t e = allow_smem(q4_down_row_kernel<6>, smem);
        if (e != cudaSuccess) return e;
        return launch(q4_down_row_kernel<6>, dim3((unsigned)p.row_tiles), dim3(32 * kRowWarps), smem, st, 0, p);
    }
    p.tiles = p.row_tiles * (c.kind == Q4_GATE_UP ? c.K : 1);
    // Warps that share a tile: those that leave the fewest chunks one after another on two CTAs an SM.
    auto steps = [&](int wk) {
        const int64_t slots = (int64_t)sms * 2 * (kRowWarps / wk);
        return (p.tiles + slots - 1) / slots * ((p.chunks + wk - 1) / wk);
    };
    p.wk = 1;
    for (int wk = 2; wk <= kRowWarps; wk *= 2)
        if (steps(wk) < steps(p.wk)) p.wk = wk;
    const int side = kRowWarps / p.wk;
    const int64_t grid = min((int64_t)(p.tiles + side - 1) / side, (int64_t)sms * 2);
    cudaError_t e;
    if (c.kind == Q4_GATE_UP) {
        if ((e = allow_smem(q4_row_kernel<2, 2>, p.vec)) != cudaSuccess) return e;
        return launch(q4_row_kernel<2, 2>, dim3((unsigned)grid), dim3(32 * kRowWarps), p.vec, st, 0, p);
    }
    if ((e = allow_smem(q4_row_kernel<1, 4>, p.vec)) != cudaSuccess) return e;
    return launch(q4_row_kernel<1, 4>, dim3((unsigned)grid), dim3(32 * kRowWarps), p.vec, st, 0, p);
}

}  // namespace q8
