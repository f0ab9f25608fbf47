// Products of 4-bit weights with several activation rows: the projection, and a chunk's experts (each expert's weights with
// the rows that chose it: gate-up with SwiGLU, and down-and-combine).
//
// A first launch lays the activation rows out as f16 parts (q4.cuh) in the order of the products' operands; a second one
// multiplies.  There a warp takes two tiles of 16 weight rows (gate-up: 16 gate rows and the 16 up rows beside them) by up
// to NT tiles of eight columns, a column being one part of one activation row.  The weights come through a ring of
// asynchronous 16-byte copies of the warp's own in shared memory, from where one matrix load gives each lane the words it
// multiplies; a block's dots are scaled by the weights' and the activation's scales into f32 sums.  What bounds it is the
// weights' bytes with few columns and the warp-wide products with many.
#include "ffn4.h"
#include "q4.cuh"

namespace q8 {
namespace {

constexpr int kWarps = 4;   // a CTA
constexpr int kStages = 6;  // of a warp's ring: chunks of four blocks of its 32 rows
constexpr int kStageBytes = 2 * 16 * 64;

struct RowsParams {
    Q4View w0, w1;
    Q4Act act;
    int64_t E, out_rows;
    int R, K;            // activation rows of the call and choices a row
    int64_t act_rows;    // rows that are laid out
    PlanPtrs plan;
    const int32_t* ids;
    const float *gates, *residual;
    uint4* parts;        // [act_rows][4 * chunks][PARTS][4]
    float* scales;       // [act_rows][4 * chunks]
    float* y;
    int64_t y_stride;
    float* out;          // down: [R * K][out_rows]
    int chunks, wk, row_tiles;
};

template <int PARTS>
__global__ void __launch_bounds__(256) q4_parts_kernel(const RowsParams p) {
    griddep_launch();
    const int octets = 16 * p.chunks;
    const int64_t n = p.act_rows * octets, step = (int64_t)gridDim.x * blockDim.x;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < ((n + 31) & ~int64_t(31)); i += step) {
        const int64_t r = min(i / octets, p.act_rows - 1);
        const int o = i < n ? (int)(i - r * octets) : octets;  // (past the end: whole warps take part)
        const ActParts a = act_parts(p.act, r, o, p.w0.cols);
        if (i >= n) continue;
        uint4* at = p.parts + (r * octets + (o & ~3)) * PARTS + (o & 3);
        at[0] = a.hi;
        if (PARTS == 2) at[4] = a.lo;
        if ((o & 3) == 0) p.scales[r * (octets / 4) + (o >> 2)] = a.scale;
    }
}

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool in) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}

__device__ __forceinline__ void load_matrices(uint32_t (&m)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(m[0]), "=r"(m[1]), "=r"(m[2]), "=r"(m[3]) : "r"(at) : "memory");
}

// d = a b, without an addend.
__device__ __forceinline__ void mma16_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                            uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
                 : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

template <int KIND, int PARTS, int NT>
__global__ void __launch_bounds__(32 * kWarps, 4) q4_rows_kernel(const RowsParams p) {
    constexpr int COLS = 8 / PARTS;  // activation rows a tile of columns
    constexpr int NC = NT * COLS;
    constexpr int AC = 4 / PARTS;    // sums a lane keeps of a tile: of rows g and g + 8, for its one or two activation rows
    extern __shared__ __align__(128) char smem[];
    __shared__ int cols[NC];  // the choices (dense: activation rows) of the columns, -1: none
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int side = kWarps / p.wk, tile = blockIdx.x * side + w / p.wk;
    const int nb = p.w0.cols >> 5, ngroups = p.w0.cols >> p.w0.group_log2;
    const int mine = (p.chunks + p.wk - 1) / p.wk, c0 = (w % p.wk) * mine, c1 = min(c0 + mine, p.chunks);
    const uint32_t ring = (uint32_t)__cvta_generic_to_shared(smem) + w * kStages * kStageBytes;
    const int total = p.R * p.K;
    bool ready = false;
    griddep_launch();
    int groups = 1;
    if (KIND != Q4_DENSE) groups = min(max(p.plan.active[0], 0), (int)min(p.E, (int64_t)total));
    for (int a = blockIdx.y; a < groups; a += gridDim.y) {
        int e = 0, first = 0, count = p.R;
        if (KIND != Q4_DENSE) {
            e = p.plan.active[1 + a];
            if (e < 0 || e >= p.E) continue;
            first = max(p.plan.offsets[e], 0);
            count = min(p.plan.offsets[e + 1], total) - first;
        }
        // the lane's rows of the two weight tiles: m-tile 0 and 1, rows g and g + 8; copies clamp to the group's last row
        const int64_t base = (int64_t)e * p.out_rows;
        const int r0 = (KIND == Q4_GATE_UP ? 16 : 32) * tile;
        const int last = (int)p.out_rows - 1;
        const uint8_t* src[2][2];
        int64_t sg[2][2];
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = min(r0 + (KIND == Q4_GATE_UP ? 0 : 16 * m) + g + 8 * i, last);
                const Q4View& v = KIND == Q4_GATE_UP && m == 1 ? p.w1 : p.w0;
                src[m][i] = v.q + (base + r) * (p.w0.cols >> 1) + 16 * t;
                sg[m][i] = (base + r) * ngroups;
            }
        for (int ct = blockIdx.z; ct * NC < count; ct += gridDim.z) {
            uint32_t into = ring;
            auto fetch = [&](int c) {  // the warp's chunk c into the next stage
                if (c < c1) {
                    const uint32_t at = into;
                    const bool in = 4 * c + t < nb;
#pragma unroll
                    for (int m = 0; m < 2; ++m)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int r = g + 8 * i;
                            copy16(at + m * 1024 + r * 64 + ((t ^ ((r >> 1) & 3)) << 4), in ? src[m][i] + 64 * c : p.w0.q, in);
                        }
                }
                asm volatile("cp.async.commit_group;" ::: "memory");
                into += kStageBytes;
                if (into == ring + kStages * kStageBytes) into = ring;
            };
            uint32_t s[2][2], z[2][2];  // the next chunk's scales and zero points: lane t block t's
            auto scales = [&](int c) {
                const int b = 4 * c + t;
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const Q4View& v = KIND == Q4_GATE_UP && m == 1 ? p.w1 : p.w0;
                        const int64_t at = sg[m][i] + ((32 * b) >> p.w0.group_log2);
                        const bool in = c < c1 && b < nb;
                        s[m][i] = in ? __ldg(v.s + at) : 0u;
                        z[m][i] = in && v.z ? __ldg(v.z + at) : 8u;
                    }
            };
#pragma unroll
            for (int i = 0; i < kStages - 1; ++i) fetch(c0 + i);
            scales(c0);
            __syncthreads();  // (the columns before these have been used)
            if (threadIdx.x < NC) {
                const int i = ct * NC + threadIdx.x;
                int c = i < count ? (KIND == Q4_DENSE ? i : p.plan.lists[first + i]) : -1;
                if (c < 0 || c >= total) c = -1;
                cols[threadIdx.x] = c;
            }
            __syncthreads();
            if (!ready) griddep_wait(), ready = true;  // the activation parts
            const int tiles = min((count - ct * NC + COLS - 1) / COLS, NT);
            // operands: column g of tile n is part g % PARTS of row g / PARTS; scales: of the rows whose sums the lane keeps
            uint32_t boff[NT], soff[NT][2 / PARTS];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const int c = max(cols[n * COLS + g / PARTS], 0);
                const uint32_t row = KIND == Q4_GATE_UP ? c / p.K : c;
                boff[n] = row * (uint32_t)(16 * p.chunks * PARTS) + (PARTS == 2 ? (g & 1) * 4 : 0) + t;
#pragma unroll
                for (int j = 0; j < 2 / PARTS; ++j) {
                    const int c2 = max(cols[n * COLS + (2 / PARTS) * t + j], 0);
                    soff[n][j] = (KIND == Q4_GATE_UP ? c2 / p.K : c2) * (uint32_t)(4 * p.chunks);
                }
            }
            float acc[2][NT][AC] = {};
            uint32_t at = ring;
            for (int c = c0; c < c1; ++c, at = at + kStageBytes == ring + kStages * kStageBytes ? ring : at + kStageBytes) {
                asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
                __syncwarp();
                fetch(c + kStages - 1);
                uint32_t sz[2][2];
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int i = 0; i < 2; ++i) sz[m][i] = s[m][i] | z[m][i] << 16;
                scales(c + 1);
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    uint32_t words[2][4];  // [m][block 2 half, rows g; rows g + 8; block 2 half + 1, rows g; rows g + 8]
#pragma unroll
                    for (int m = 0; m < 2; ++m) {
                        const int r = (lane & 7) + (lane & 8), b = 2 * half + (lane >> 4);
                        load_matrices(words[m], at + m * 1024 + r * 64 + ((b ^ ((r >> 1) & 3)) << 4));
                    }
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const int b = 2 * half + k;
                        uint32_t h[2][2][4];
                        float sw[2][2];
#pragma unroll
                        for (int m = 0; m < 2; ++m)
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                const uint32_t v = __shfl_sync(0xffffffffu, sz[m][i], (lane & ~3) + b);
                                uint32_t zc, zf;
                                zero_forms(v >> 16, zc, zf);
                                words_f16(words[m][2 * k + i], zc, zf, h[m][i]);
                                sw[m][i] = scale_f32(v & 0xffffu, p.w0.bf16);
                            }
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            if (n < tiles) {
                                const uint4 x = __ldca(p.parts + boff[n] + (uint32_t)(4 * c + b) * (4 * PARTS));
                                float sx[2 / PARTS];
#pragma unroll
                                for (int j = 0; j < 2 / PARTS; ++j) sx[j] = __ldca(p.scales + soff[n][j] + 4 * c + b);
#pragma unroll
                                for (int m = 0; m < 2; ++m) {
                                    float d[4];
                                    mma16_first(d, h[m][0][0], h[m][1][0], h[m][0][1], h[m][1][1], x.x, x.y);
                                    mma16(d, h[m][0][2], h[m][1][2], h[m][0][3], h[m][1][3], x.z, x.w);
                                    if (PARTS == 2) {
                                        acc[m][n][0] = fmaf(sw[m][0] * sx[0], d[0] + d[1], acc[m][n][0]);
                                        acc[m][n][1] = fmaf(sw[m][1] * sx[0], d[2] + d[3], acc[m][n][1]);
                                    } else {
#pragma unroll
                                        for (int j = 0; j < 4; ++j)
                                            acc[m][n][j % AC] = fmaf(sw[m][j >> 1] * sx[(j & 1) % (2 / PARTS)], d[j], acc[m][n][j % AC]);
                                    }
                                }
                            }
                        }
                    }
                }
            }
            asm volatile("cp.async.wait_group 0;" ::: "memory");
            if (p.wk > 1) {  // the warps' sums of the tile's columns, in their order
                __syncthreads();
                float* red = reinterpret_cast<float*>(smem);
                if (w % p.wk) {
#pragma unroll
                    for (int m = 0; m < 2; ++m)
#pragma unroll
                        for (int n = 0; n < NT; ++n)
#pragma unroll
                            for (int j = 0; j < AC; ++j) red[(w * (2 * NT * AC) + (m * NT + n) * AC + j) * 32 + lane] = acc[m][n][j];
                }
                __syncthreads();
                if (w % p.wk == 0) {
                    for (int k = 1; k < p.wk; ++k)
#pragma unroll
                        for (int m = 0; m < 2; ++m)
#pragma unroll
                            for (int n = 0; n < NT; ++n)
#pragma unroll
                                for (int j = 0; j < AC; ++j)
                                    acc[m][n][j] += red[((w + k) * (2 * NT * AC) + (m * NT + n) * AC + j) * 32 + lane];
                }
            }
            if (w % p.wk == 0 && tile < p.row_tiles) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int j = 0; j < AC; ++j) {
                        // PARTS 2: j is the row half; PARTS 1: j is row half * 2 + activation row
                        const int i = PARTS == 2 ? j : j >> 1;
                        const int c = cols[n * COLS + (2 / PARTS) * t + (PARTS == 2 ? 0 : j & 1)];
                        if (c < 0) continue;
                        const int r = r0 + g + 8 * i;
                        if (KIND == Q4_GATE_UP) {
                            if (r <= last) p.y[c * p.y_stride + r] = silu_f32(acc[0][n][j]) * acc[1][n][j];
                        } else {
                            float* to = KIND == Q4_DENSE ? p.y + c * p.y_stride : p.out + c * p.out_rows;
                            if (r <= last) to[r] = acc[0][n][j];
                            if (r + 16 <= last) to[r + 16] = acc[1][n][j];
                        }
                    }
            }
            if (p.wk > 1) __syncthreads();  // (the ring takes the next columns' weights)
        }
    }
    if (!ready) griddep_wait();  // (a grid ends after the launch before it, whatever its CTAs had to do)
}

// y[r] = residual[r] + sum_j gates[r][j] out[r][j], in the order of the choices.
__global__ void __launch_bounds__(256) q4_combine_kernel(const RowsParams p) {
    griddep_wait();
    const int64_t n = (int64_t)p.R * p.out_rows, step = (int64_t)gridDim.x * blockDim.x;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += step) {
        const int64_t r = i / p.out_rows, o = i - r * p.out_rows;
        float sum = 0.f;
        for (int j = 0; j < p.K; ++j) {
            const int64_t c = r * p.K + j;
            const int e = p.ids[c];
            if (e >= 0 && e < p.E) sum = fmaf(p.gates[c], p.out[c * p.out_rows + o], sum);
        }
        p.y[i] = p.residual ? p.residual[i] + sum : sum;
    }
}

template <int KIND, int PARTS, int NT>
cudaError_t run(const RowsParams& p, dim3 grid, cudaStream_t st) {
    constexpr size_t smem = (size_t)kWarps * kStages * kStageBytes;
    static_assert(smem >= (size_t)kWarps * 2 * NT * (4 / PARTS) * 128, "the warps' sums fit the ring");
    const cudaError_t e = cudaFuncSetAttribute(q4_rows_kernel<KIND, PARTS, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    return launch(q4_rows_kernel<KIND, PARTS, NT>, grid, dim3(32 * kWarps), smem, st, 1, p);
}

template <int PARTS, int NT>
cudaError_t run_kind(int kind, const RowsParams& p, dim3 grid, cudaStream_t st) {
    if (kind == Q4_DENSE) return run<Q4_DENSE, PARTS, NT>(p, grid, st);
    if (kind == Q4_GATE_UP) return run<Q4_GATE_UP, PARTS, NT>(p, grid, st);
    return run<Q4_DOWN, PARTS, NT>(p, grid, st);
}

}  // namespace

cudaError_t launch_q4_row(const Q4Call& c, cudaStream_t st);

cudaError_t launch_q4(const Q4Call& c, Carve& ws, cudaStream_t st) {
    if (c.R == 1) return launch_q4_row(c, st);
    const int parts = c.act.x || c.act.lo ? 2 : 1;
    RowsParams p = {};
    p.w0 = c.w0;
    p.w1 = c.w1;
    p.act = c.act;
    p.E = c.E;
    p.out_rows = c.out_rows;
    p.R = (int)c.R;
    p.K = c.K;
    p.act_rows = c.kind == Q4_DOWN ? c.R * c.K : c.R;
    p.plan = c.plan;
    p.ids = c.ids;
    p.gates = c.gates;
    p.residual = c.residual;
    p.y = c.y;
    p.y_stride = c.y_stride;
    p.chunks = (c.w0.cols + 127) / 128;
    p.parts = ws.take<uint4>((size_t)p.act_rows * p.chunks * 16 * parts);
    p.scales = ws.take<float>((size_t)p.act_rows * p.chunks * 4);
    if (c.kind == Q4_DOWN) p.out = ws.take<float>((size_t)c.R * c.K * c.out_rows);
    if (ws.overflow) return cudaSuccess;
    const int sms = device_info().sms;
    const int64_t octets = p.act_rows * p.chunks * 16;
    const dim3 lay((unsigned)min((octets + 255) / 256, (int64_t)sms * 8));
    cudaError_t e = parts == 2 ? launch(q4_parts_kernel<2>, lay, dim3(256), 0, st, 0, p)
                               : launch(q4_parts_kernel<1>, lay, dim3(256), 0, st, 0, p);
    if (e != cudaSuccess) return e;
    p.row_tiles = (int)((c.out_rows + (c.kind == Q4_GATE_UP ? 15 : 31)) / (c.kind == Q4_GATE_UP ? 16 : 32));
    const int64_t groups = c.kind == Q4_DENSE ? 1 : min(c.E, c.R * c.K);
    const int nc = 32;
    const int64_t zs = c.kind == Q4_DENSE ? min((c.R + nc - 1) / nc, (int64_t)65535) : 1;
    // Warps that share a tile: as many as it takes for 16 warps an SM.
    p.wk = 1;
    while (p.wk < kWarps && p.wk * 2 <= p.chunks && p.row_tiles * groups * zs * p.wk < (int64_t)sms * 16) p.wk *= 2;
    const int side = kWarps / p.wk;
    const dim3 grid((unsigned)((p.row_tiles + side - 1) / side), (unsigned)min(groups, (int64_t)65535), (unsigned)zs);
    e = parts == 2 ? run_kind<2, 8>(c.kind, p, grid, st) : run_kind<1, 4>(c.kind, p, grid, st);
    if (e != cudaSuccess || c.kind != Q4_DOWN) return e;
    const int64_t n = c.R * c.out_rows;
    return launch(q4_combine_kernel, dim3((unsigned)min((n + 255) / 256, (int64_t)sms * 16)), dim3(256), 0, st, 1, p);
}

}  // namespace q8
