// Products of 4-bit weights with one activation row: the projection, and a row's experts (gate-up with SwiGLU, and
// down-and-combine).
//
// The work is bound by the weights' bytes and, close behind, by the instructions that unpack them.  A warp takes 16 rows by
// steps of eight 32-value blocks (128 bytes a row), which come through a ring of asynchronous copies of its own; lane (g, t)
// reads whole blocks of rows g and g + 8 from it, block t of each half step.
//   - Quantized activations: integer dot products of four bytes, the zero point taken out of the block's sum by the sum of
//     the activation's words; exact.
//   - f32 activations: warp-wide f16 products (q4.cuh).  A lane's block is an A operand if the product's sum over t is kept
//     apart, which its eight columns do: column (j, p) holds part p of the activation's block j, and zeros where the lanes
//     with t != j read.  Lane (g, t) then receives the two parts' dots of its own block of its own rows.
// Either way a block's dot meets its scales in the lane that loaded them: nothing is shuffled until a tile ends, and every
// group size costs the same.
// Measured, replayed: 151936 x 2048, group 128, one-word activations 29 us (163 MB, 5.6 TB/s, 82% of the measured copy rate;
// f32 42); 5120 x 2048, f32, 5.5; eight experts of 2048 x 768 with their sum 16 (21 MB, two launches of one wave each, whose
// start, first loads and end are most of it).  Why a ring of 16-byte copies: plain 16-byte loads into registers took 55 us for
// the 29, a lane's loads in flight being bound by its registers.
#include "ffn4.h"
#include "q4.cuh"

namespace q8 {
namespace {

constexpr int kRowWarps = 8;
// Of a warp's ring.  Three leave an SM room for the next launch's CTAs beside gate-up's: eight experts of 2048 x 768 17.4 us with
// four, 15.7 with three, 15.4 with two; a long row of words needs three (151936 x 2048 29.1 and 32.4).
constexpr int kRowStages = 3;
constexpr int kStepBytes = 16 * 128;  // a step of one tile's rows

// A block of the activation in shared memory.  f32: two parts of 64 bytes, and 16 more so that four blocks lie in different
// banks (its unit stands in the array behind, as two factors).  Words: 32 bytes (and 32 of low words), then scale and sum.
template <int FORM>
constexpr int block_bytes() { return FORM == FORM_F32 ? 144 : FORM == FORM_ONE ? 48 : 80; }

struct RowParams {
    Q4View w0, w1;
    Q4Act act;
    int kind;
    int64_t E, out_rows;  // rows a group
    int K;
    const int32_t* ids;
    const float *gates, *residual;
    float* y;
    int steps;            // of a row
    int parts_log2;       // warps' parts of a row's steps
    int segs, spw, side;  // a tile's segments (parts, or experts times parts), those a warp takes, tiles side by side
    int tiles;            // of 16 rows, of a choice's for gate-up
    int vecs;             // activation rows
    uint32_t vec;         // bytes of one in shared memory
};

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// The activation's rows in shared memory, zeros up to whole steps.
template <int FORM>
__device__ __forceinline__ void stage_rows(const RowParams& p, char* vecs) {
    const int octets = 32 * p.steps, cols = p.w0.cols;  // eight values each
    for (int i = threadIdx.x; i < p.vecs * octets; i += blockDim.x) {  // whole warps, a block's four lanes together
        const int v = i / octets, o = i - v * octets, b = o >> 2;
        char* at = vecs + v * p.vec + b * block_bytes<FORM>();
        if (FORM == FORM_F32) {
            float x[8];
            act_values(p.act, v, o, cols, x);
            float m = finite_max(x);
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
            const ActParts a = split_values(x, m);
            *reinterpret_cast<uint4*>(at + (o & 3) * 16) = a.hi;
            *reinterpret_cast<uint4*>(at + 64 + (o & 3) * 16) = a.lo;
            // The unit 2^k as 2^(k >> 1) for the weights' scale and the rest for the dot: with the whole of it on the scale their
            // product left f32's range below long before the block's result did.
            const int k = (int)(__float_as_uint(a.scale) >> 23) - 127, half = k >> 1;
            if ((o & 3) == 0)
                *reinterpret_cast<float2*>(vecs + v * p.vec + 8 * p.steps * 144 + 8 * b) =
                    make_float2(__int_as_float((127 + half) << 23), __int_as_float((127 + k - half) << 23));
        } else {
            const int64_t from = (int64_t)v * cols + 8 * o;
            const bool in = 8 * o < cols;
            int sum = 0;
#pragma unroll
            for (int k = 0; k < (FORM == FORM_TWO ? 2 : 1); ++k) {
                const uint2 x = in ? *reinterpret_cast<const uint2*>((k ? p.act.lo : p.act.q) + from) : make_uint2(0, 0);
                sum = sum * 128 + __dp4a((int)x.x, 0x01010101, __dp4a((int)x.y, 0x01010101, 0));
                *reinterpret_cast<uint2*>(at + 32 * k + (o & 3) * 8) =
                    make_uint2(__byte_perm(x.x, x.y, 0x6420), __byte_perm(x.x, x.y, 0x7531));  // even values, odd values
            }
            sum += __shfl_xor_sync(0xffffffffu, sum, 1);
            sum += __shfl_xor_sync(0xffffffffu, sum, 2);
            if ((o & 3) == 0) {
                float scale = in ? p.act.s[from >> 5] : 0.f;
                if (FORM == FORM_TWO) scale *= 0.0078125f;
                *reinterpret_cast<float2*>(at + (FORM == FORM_TWO ? 64 : 32)) = make_float2(scale, __int_as_float(sum));
            }
        }
    }
}

__device__ __forceinline__ uint32_t word_of(const uint4& v, int m) { return m == 0 ? v.x : m == 1 ? v.y : m == 2 ? v.z : v.w; }

// An activation block as the lane multiplies it.
template <int FORM>
struct Operand {
    uint4 v[FORM == FORM_F32 || FORM == FORM_TWO ? 4 : 2];
    float scale, rest;  // f32: the unit is their product
    int sum;
};

// acc[i] += block t of row g + 8 i (words w[i], scale sw[i], zero point z[i]) times the activation's.
template <int FORM>
__device__ __forceinline__ void multiply(const uint4 (&w)[2], const float (&sw)[2], const uint32_t (&z)[2], const Operand<FORM>& x,
                                         float (&acc)[2]) {
    if (FORM == FORM_F32) {
        float d[4] = {0.f, 0.f, 0.f, 0.f};
        uint32_t zc[2], zf[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) zero_forms(z[i], zc[i], zf[i]);
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            uint32_t h0[4], h1[4];
            words_f16(word_of(w[0], m), zc[0], zf[0], h0);
            words_f16(word_of(w[1], m), zc[1], zf[1], h1);
            mma16(d, h0[0], h1[0], h0[1], h1[1], x.v[m].x, x.v[m].y);
            mma16(d, h0[2], h1[2], h0[3], h1[3], x.v[m].z, x.v[m].w);
        }
        acc[0] = fmaf(sw[0] * x.scale, (d[0] + d[1]) * x.rest, acc[0]);
        acc[1] = fmaf(sw[1] * x.scale, (d[2] + d[3]) * x.rest, acc[1]);
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            int hi = 0, lo = 0;
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const uint32_t u = word_of(w[i], m);
                const int even = u & 0x0f0f0f0f, odd = (u >> 4) & 0x0f0f0f0f;
                const uint4 v = x.v[m >> 1];
                hi = __dp4a(odd, (int)(m & 1 ? v.w : v.y), __dp4a(even, (int)(m & 1 ? v.z : v.x), hi));
                if (FORM == FORM_TWO) {
                    const uint4 l = x.v[(FORM == FORM_TWO ? 2 : 0) + (m >> 1)];
                    lo = __dp4a(odd, (int)(m & 1 ? l.w : l.y), __dp4a(even, (int)(m & 1 ? l.z : l.x), lo));
                }
            }
            if (FORM == FORM_TWO) hi = hi * 128 + lo;
            hi -= (int)z[i] * x.sum;
            acc[i] = fmaf(sw[i] * x.scale, (float)hi, acc[i]);
        }
    }
}

__device__ __forceinline__ float quad_sum(float v) {
    v += __shfl_xor_sync(0xffffffffu, v, 1);
    return v + __shfl_xor_sync(0xffffffffu, v, 2);
}

// A CTA takes `side` tiles at a time (all of a tile's segments), its warps their segments' steps one after another over all
// their tiles.  MT = 2 (gate-up): a tile is 16 gate rows and the 16 up rows beside them.
template <int FORM, int MT>
__global__ void __launch_bounds__(32 * kRowWarps, 2) q4_row_kernel(const RowParams p) {
    extern __shared__ __align__(128) char smem[];
    __shared__ uint4 zeros[4];
    const bool has_z = p.w0.z != nullptr;
    griddep_wait();  // (launches overlap up to here: nothing is read before the launch before has ended)
    griddep_launch();
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int nb = p.w0.cols >> 5, last = (int)p.out_rows - 1, choice = blockIdx.y;  // gate-up: the CTA's choice
    const int64_t row_bytes = p.w0.cols >> 1;
    const int row_groups = p.w0.cols >> p.w0.group_log2, mine = (p.steps + (1 << p.parts_log2) - 1) >> p.parts_log2;
    const int own_seg = p.side > 1 ? w & (p.segs - 1) : w, off_tile = p.side > 1 ? w / p.segs : 0;
    const int stride = gridDim.x * p.side, first = off_tile < p.side ? (int)blockIdx.x * p.side + off_tile : p.tiles;
    const int rounds = (p.tiles - (int)blockIdx.x * p.side + stride - 1) / stride;  // the CTA's, alike in all its warps
    char* ring = smem + w * (kRowStages * MT * kStepBytes);
    char* vecs = smem + kRowWarps * kRowStages * MT * kStepBytes;
    float* part = reinterpret_cast<float*>(vecs + p.vecs * p.vec);  // [2][side * segs][MT][16]
    const int slots = p.side * p.segs;
    auto expert = [&](int j) {  // of the row's choice j, or -1
        const int e = p.ids ? p.ids[j] : 0;
        return e >= 0 && e < p.E ? e : -1;
    };

    // A place in the warp's run of (tile, segment, step).
    struct Place {
        int tile, seg, at, step;  // step: the first of the segment, then the next one
        int64_t row;              // the lane's row g (less where the tile ends), -1: none
        int more;                 // rows from there to row g + 8
    };
    auto locate = [&](Place& l) {
        l.at = 0;
        l.row = -1;
        l.step = (l.seg & ((1 << p.parts_log2) - 1)) * mine;
        if (l.tile >= p.tiles || l.seg >= p.segs) return;
        const int e = expert(p.kind == Q4_DOWN ? l.seg >> p.parts_log2 : choice), r0 = 16 * l.tile + g;
        if (e < 0) return;
        l.row = e * p.out_rows + min(r0, last);
        l.more = min(r0 + 8, last) - min(r0, last);
    };
    auto advance = [&](Place& l) {
        ++l.step;
        if (++l.at < mine) return;
        l.seg += kRowWarps;
        if (p.spw == 1 || l.seg >= p.spw * kRowWarps) l.seg = own_seg, l.tile += stride;
        locate(l);
    };
    Place in = {first, own_seg}, sc = in;
    locate(in);
    sc = in;
    // copies: 16-byte unit u of a row of the step stands at u ^ 4 (row & 1), so that two rows' units lie in different banks
    const uint32_t to = (uint32_t)__cvta_generic_to_shared(ring) + g * 128 + ((t ^ (4 * (g & 1))) << 4);
    uint32_t into = 0;
    auto fetch = [&]() {
        if (in.row >= 0 && in.step < p.steps) {
            const int64_t from = in.row * row_bytes + 128 * in.step + 16 * t, more = in.more * row_bytes;
            const bool one = 8 * in.step + t < nb, two = 8 * in.step + 4 + t < nb;
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const uint8_t* a = (m ? p.w1.q : p.w0.q) + from;
                const uint32_t d = to + into + m * kStepBytes;
                if (one) copy16(d, a), copy16(d + 1024, a + more);
                if (two) copy16(d ^ 64, a + 64), copy16((d + 1024) ^ 64, a + more + 64);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        into = into == (kRowStages - 1) * MT * kStepBytes ? 0 : into + MT * kStepBytes;
        advance(in);
    };
    uint32_t s[MT][2][2], z[MT][2][2];  // the next step's scales and zero points: [half step][row g, g + 8]
    auto scales = [&]() {
        const bool ok = sc.row >= 0 && sc.step < p.steps;
        const int64_t row = sc.row * row_groups;
        const int more = sc.more * row_groups;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int b = 8 * sc.step + 4 * k + t, col = (32 * b) >> p.w0.group_log2;
            const bool here = ok && b < nb;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int64_t at = row + (i ? col + more : col);
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    s[m][k][i] = here ? __ldg((m ? p.w1.s : p.w0.s) + at) : 0u;
                    if (has_z) z[m][k][i] = here ? __ldg((m ? p.w1.z : p.w0.z) + at) : 8u;
                }
            }
        }
        advance(sc);
    };
#pragma unroll
    for (int i = 0; i < kRowStages - 1; ++i) fetch();
    scales();
    if (threadIdx.x < 4) zeros[threadIdx.x] = make_uint4(0, 0, 0, 0);
    stage_rows<FORM>(p, vecs);
    __syncthreads();
    const bool own = (g >> 1) == t;  // f32: the lane holds a column of its own block
    uint32_t from = 0;
    int buf = 0;
    for (int round = 0; round < rounds; ++round, buf ^= 1) {
        const int tile = first + round * stride;
        for (int k = 0; k < p.spw; ++k) {
            const int seg = own_seg + k * kRowWarps;
            const bool real = off_tile < p.side && seg < p.segs;
            const int step0 = (seg & ((1 << p.parts_log2) - 1)) * mine;
            const char* vec = vecs + (p.kind == Q4_DOWN && real ? seg >> p.parts_log2 : 0) * p.vec;
            float acc[MT][2] = {};
            for (int i = 0; i < mine; ++i) {
                asm volatile("cp.async.wait_group %0;" ::"n"(kRowStages - 2) : "memory");
                __syncwarp();
                fetch();
                const int step = step0 + i;
                float sw[MT][2][2];
                uint32_t zz[MT][2][2];
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int j = 0; j < 2; ++j) sw[m][h][j] = scale_f32(s[m][h][j], p.w0.bf16), zz[m][h][j] = has_z ? z[m][h][j] : 8u;
                scales();
                if (real && step < p.steps) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int b = 8 * step + 4 * h + t;
                        Operand<FORM> x;
                        if (FORM == FORM_F32) {
                            const char* at = own ? vec + b * 144 + (g & 1) * 64 : reinterpret_cast<const char*>(zeros);
#pragma unroll
                            for (int m = 0; m < 4; ++m) x.v[m] = *reinterpret_cast<const uint4*>(at + 16 * m);
                            const float2 f = *reinterpret_cast<const float2*>(vec + 8 * p.steps * 144 + 8 * b);
                            x.scale = f.x, x.rest = f.y;
                        } else {
                            const char* at = vec + b * block_bytes<FORM>();
#pragma unroll
                            for (int m = 0; m < (FORM == FORM_TWO ? 4 : 2); ++m) x.v[m] = *reinterpret_cast<const uint4*>(at + 16 * m);
                            const float2 f = *reinterpret_cast<const float2*>(at + (FORM == FORM_TWO ? 64 : 32));
                            x.scale = f.x, x.sum = __float_as_int(f.y);
                        }
#pragma unroll
                        for (int m = 0; m < MT; ++m) {
                            const char* at = ring + from + m * kStepBytes + g * 128 + (((t + 4 * h) ^ (4 * (g & 1))) << 4);
                            const uint4 words[2] = {*reinterpret_cast<const uint4*>(at), *reinterpret_cast<const uint4*>(at + 1024)};
                            multiply<FORM>(words, sw[m][h], zz[m][h], x, acc[m]);
                        }
                    }
                }
                from = from == (kRowStages - 1) * MT * kStepBytes ? 0 : from + MT * kStepBytes;
            }
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float v = quad_sum(acc[m][i]);
                    if (t == 0 && real) part[((buf * slots + off_tile * p.segs + seg) * MT + m) * 16 + g + 8 * i] = v;
                }
        }
        __syncthreads();  // (the next tiles' sums go to the other half: one barrier a round)
        if (own_seg == 0 && lane < 16 && tile < p.tiles) {
            const float* sums = part + (buf * slots + off_tile * p.segs) * MT * 16 + lane;
            const int r = 16 * tile + lane;
            if (p.kind == Q4_DOWN) {
                float sum = 0.f;
                for (int j = 0; j < p.K; ++j) {
                    if (expert(j) < 0) continue;
                    float v = 0.f;
                    for (int i = 0; i < 1 << p.parts_log2; ++i) v += sums[((j << p.parts_log2) + i) * 16];
                    sum = fmaf(p.gates[j], v, sum);
                }
                if (r <= last) p.y[r] = p.residual ? p.residual[r] + sum : sum;
            } else {
                float v[MT] = {};
                for (int i = 0; i < p.segs; ++i)
#pragma unroll
                    for (int m = 0; m < MT; ++m) v[m] += sums[(i * MT + m) * 16];
                if (r <= last && expert(choice) >= 0) p.y[choice * p.out_rows + r] = MT == 2 ? silu_f32(v[0]) * v[MT - 1] : v[0];
            }
        }
    }
}

constexpr size_t kRowSmem = 220 << 10;

size_t row_smem(const RowParams& p, int mt) {
    return (size_t)kRowWarps * kRowStages * mt * kStepBytes + (size_t)p.vecs * p.vec + 2 * (size_t)p.side * p.segs * mt * 64;
}

// How a tile's steps are dealt to the warps: 2^parts_log2 parts of a row each (of an expert's, for down).
void deal(RowParams& p, int parts_log2) {
    p.parts_log2 = parts_log2;
    p.segs = (p.kind == Q4_DOWN ? p.K : 1) << parts_log2;
    p.spw = (p.segs + kRowWarps - 1) / kRowWarps;
    p.side = p.spw > 1 || p.kind == Q4_DOWN ? 1 : kRowWarps / p.segs;
}

template <int FORM, int MT>
cudaError_t run(const RowParams& p, cudaStream_t st) {
    const size_t smem = row_smem(p, MT);
    static std::atomic<uint64_t> done;
    const cudaError_t e = allow_smem(q4_row_kernel<FORM, MT>, kRowSmem, done);
    if (e != cudaSuccess) return e;
    const int choices = p.kind == Q4_GATE_UP ? p.K : 1;
    const int64_t ctas = (p.tiles + p.side - 1) / p.side, most = max(device_info().sms * 2 / choices, 1);
    return launch(q4_row_kernel<FORM, MT>, dim3((unsigned)min(ctas, most), choices), dim3(32 * kRowWarps), smem, st, 1, p);
}

template <int FORM>
cudaError_t run_kind(RowParams p, cudaStream_t st) {
    p.vec = (uint32_t)(8 * p.steps * (block_bytes<FORM>() + (FORM == FORM_F32 ? 8 : 0)));
    // The parts that leave an SM the fewest steps, counting half a one for each tile's end.  Measured, us, 1, 2, 4 and 8 parts, f32:
    // 2048 x 4096 13.3, 8.3, 5.7 and 4.3; 8192 x 4096 13.3, 8.3, 8.1 and 8.5; 151936 x 2048 42, 44, 49 and 57.
    int best = 0;
    int64_t fewest = INT64_MAX;
    for (int l = 0; l <= 3 && (1 << l) <= p.steps; ++l) {
        deal(p, l);
        const int64_t ctas = (int64_t)(p.tiles + p.side - 1) / p.side * (p.kind == Q4_GATE_UP ? p.K : 1), sms = device_info().sms;
        const int64_t steps = (ctas + sms - 1) / sms * (2 * p.spw * ((p.steps + (1 << l) - 1) >> l) + 1);
        if (steps < fewest) fewest = steps, best = l;
    }
    deal(p, best);
    return p.kind == Q4_GATE_UP ? run<FORM, 2>(p, st) : run<FORM, 1>(p, st);
}

}  // namespace

// Whether the row's activations fit a CTA (an expert's hidden rows may be many and long).
bool q4_row_fits(const Q4Call& c) {
    const size_t steps = (c.w0.cols + 255) / 256, vecs = c.kind == Q4_DOWN ? c.K : 1;
    const size_t block = c.act.x ? 152 : c.act.lo ? 80 : 48;
    const size_t mt = c.kind == Q4_GATE_UP ? 2 : 1, segs = 8 * vecs;
    return (size_t)kRowWarps * kRowStages * mt * kStepBytes + vecs * steps * 8 * block + 2 * segs * mt * 64 <= kRowSmem;
}

cudaError_t launch_q4_row(const Q4Call& c, cudaStream_t st) {
    RowParams p = {};
    p.w0 = c.w0;
    p.w1 = c.w1;
    p.act = c.act;
    p.kind = c.kind;
    p.E = c.E;
    p.out_rows = c.out_rows;
    p.K = c.K;
    p.ids = c.kind == Q4_DENSE ? nullptr : c.ids;
    p.gates = c.gates;
    p.residual = c.residual;
    p.y = c.y;
    p.steps = (c.w0.cols + 255) / 256;
    p.vecs = c.kind == Q4_DOWN ? c.K : 1;
    p.tiles = (int)((c.out_rows + 15) / 16);
    if (c.act.x) return run_kind<FORM_F32>(p, st);
    return c.act.lo ? run_kind<FORM_TWO>(p, st) : run_kind<FORM_ONE>(p, st);
}

}  // namespace q8
