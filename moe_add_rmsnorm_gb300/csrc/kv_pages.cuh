// Device helpers of the paged, quantized key/value cache: which sequence a row belongs to, where a position lives, and
// the 8-bit words' values.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "kernels.h"
#include "q8moe.h"

namespace q8 {

// One sequence of a batch.  `rows_ok`: its rows lie within the call's; `len_ok`: its length holds its rows and fits the
// page table.
struct KvSeq {
    int64_t first = 0, n = 0;
    int len = 0;
    bool rows_ok = false, len_ok = false;
    // Whether row r is the sequence's and has a position (a row_start that decreases leads rows to sequences not theirs).
    __device__ bool holds(int64_t r) const { return rows_ok && len_ok && r >= first && r < first + n; }
};

__device__ __forceinline__ KvSeq kv_seq(const KvView& p, int b) {
    KvSeq s;
    s.first = __ldg(p.row_start + b);
    s.n = (int64_t)__ldg(p.row_start + b + 1) - s.first;
    s.len = __ldg(p.kv_len + b);
    s.rows_ok = s.first >= 0 && s.n >= 0 && s.first + s.n <= p.rows;
    s.len_ok = s.len >= s.n && s.len <= p.cap;
    return s;
}

__device__ __forceinline__ void kv_flag(const KvView& p, int bit) {
    if (p.error) atomicOr(p.error, bit);
}

// Records a batch's sequences whose rows are not the call's or whose length is out of range, whether a row of the call leads
// to them or not: for a CTA of 256 threads of its own, beside those that take the rows (launched where there is an error word).
__device__ __forceinline__ void kv_check(const KvView& p) {
    bool bad = false;
#pragma unroll 4
    for (int b = threadIdx.x; b < p.seqs; b += Q8_THREADS) {  // (without the flag inside: several loads at once)
        const KvSeq s = kv_seq(p, b);
        bad |= !s.rows_ok || (s.n > 0 && !s.len_ok);
    }
    if (bad) kv_flag(p, Q8_KV_ERR_LENGTH);
}

// The sequence row r belongs to, or -1 (all lanes of a warp call it with the same r).  A 32-way search for the last b
// with row_start[b] <= r: every step leaves at most a 32nd of the range, so 32 sequences take one round of loads.
__device__ __forceinline__ int kv_find_seq(const KvView& p, int64_t r) {
    const int lane = threadIdx.x & 31;
    int lo = 0, n = p.seqs + 1;
    while (n > 0) {
        const int step = (n + 31) / 32, i = lane * step + step - 1;
        const unsigned below = __ballot_sync(0xffffffffu, i < n && __ldg(p.row_start + lo + (i < n ? i : 0)) <= r);
        const int c = __popc(below) * step;
        lo += c;
        n = min(n - c, step - 1);
    }
    return lo - 1 < p.seqs ? lo - 1 : -1;
}

// The page of position `pos` of sequence b, or -1 when its id is out of range (pos within the table).
__device__ __forceinline__ int kv_page(const KvView& p, int b, int pos) {
    const int id = __ldg(p.table + b * p.table_stride + (pos >> p.page_log2));
    return id >= 0 && id < p.pages ? id : -1;
}

// The index of a cached row: its scale's, and its words' divided by head_dim.
__device__ __forceinline__ int64_t kv_row(const KvView& p, int page, int head, int pos) {
    return (((int64_t)page * p.kv + head) << p.page_log2) + (pos & ((1 << p.page_log2) - 1));
}

// Two e4m3 words (the low and the high byte of w) as two f16 values in one register (exact).
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t w) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(w));
    return h;
}

}  // namespace q8
