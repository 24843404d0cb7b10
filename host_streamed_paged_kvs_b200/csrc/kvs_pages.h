// kvs_pages.h -- arguments and launchers of the batch operators over
// caller-owned pages (append, read-back, attention), shared by their host
// entry points (kvs_pages.cpp) and kernels.  Not part of the public ABI.
#pragma once

#include "kvs_internal.h"

namespace kvs {

// value types of K, V, Q and outputs (the public KVS_DT_* codes)
enum : int { kDtF16 = 0, kDtBF16 = 1, kDtF32 = 2 };

struct PagePool {
    uint8_t* pages;
    int n_pages, n_kv;
    int k_type, v_type;
};

struct PageBatch {
    int n_seqs, n_rows;
    const int* q_start;
    const int* seq_len;
    const int* table;
    int table_stride;
    int* status;
};

// a [rows][heads][128] tensor, strides in values
struct RowsRef {
    void* p;
    long long row, head;
};

struct AppendPagesArgs {
    PagePool pool;
    PageBatch batch;
    RowsRef k, v, q, q_out;
    int n_qh;               // 0 = no Q
    const float* inv_freq;  // null = no rotation
    int rot;                // rotated dims of a head
    int interleaved;
    const int* positions;
    int pos_offset;
    float mscale;
};

struct ReadPagesArgs {
    PagePool pool;
    PageBatch batch;
    RowsRef k, v;  // p null = not wanted
};

// Attention of the batch.  Rows of one kv head are the pairs (token, head of the
// group), token-major.  A call runs one or two phases: the prefix phase (every
// row against the shared prefix, results kept as one record per row in prior_*)
// and the own phase (each sequence's rows against its own pages, joined with
// prior_* where there is a prefix).
struct AttendPagesArgs {
    PagePool pool;
    PageBatch batch;
    int n_qh, group;
    RowsRef q, out;
    int q_dtype, out_dtype;
    float* lse;              // [n_rows][n_qh] or null
    float scale, softcap;    // natural units; softcap 0 = none
    float inv_cap;           // 1 / softcap
    int window;
    const float* slopes;
    const int* first_key;
    const int* end_key;
    const int* prefix_table;
    int prefix_len;
    int prefix_phase;        // 1: keys are the prefix's, results go to prior_*
    int precise;             // probabilities as two fp16 terms
    float* prior_acc;        // [n_rows][n_qh][128], relative to 2^ref
    float2* prior_ml;        // [n_rows][n_qh] (ref, sum)
    float* records;          // pieces of units that several CTAs share
    int* counters;           // arrivals at such a unit, zero between calls
    int few_rows;            // own phase: sequences with more rows per kv head than this belong
                             // to the many-row kernel, the others to the few-row one
    struct WideUnit* units;  // the many-row kernel's list, made on the device for each call
    struct WidePlan* plan;
};

// One row group (up to 256 rows of a sequence, or of the batch) and the 128-key
// stages it needs; each kv head has a unit of it.
struct WideUnit {
    int seq, row0, rows;     // rows row0 .. row0 + rows - 1 of the sequence, token-major
    int stage0, n_stages;    // at least 1
    int n_keys;              // keys that exist; 0 where no row sees any
    long long before;        // length of the groups before this one in the list
};
struct WidePlan {
    int n_groups, pad;
    long long total;         // length of all groups in the list
};
constexpr int kWideRows = 256;
constexpr int kWideCtas = 148;
constexpr size_t kWideRecordBytes = (size_t)kWideCtas * 2 * kWideRows * 132 * 4;
// groups of a batch: full ones and one ragged end per sequence
inline long long wide_groups(long long n_rows, int group, long long n_seqs) {
    return n_rows * group / kWideRows + n_seqs + 1;
}

// a unit of the few-row kernel has 8 or 16 rows; a sequence of up to 32 rows is one or two units
constexpr int kFewRowsMax = 16;
constexpr int kFewSeqRows = 32;
constexpr int kRecordFloats = 132;      // 128 sums, reference, sum of weights, padding
constexpr int kFewCtas = 296;           // two per SM
constexpr size_t kFewRecordBytes = (size_t)kFewCtas * 2 * kFewRowsMax * kRecordFloats * 4;

struct PageMaps {
    CUtensorMap k, v;  // K and V codes as boxes of 128 tokens
};

cudaError_t launch_attend_few(const AttendPagesArgs& a, const PageMaps& maps, int unit_rows, int n_sms, cudaStream_t s);

cudaError_t launch_attend_wide(const AttendPagesArgs& a, const PageMaps& maps, int n_sms, cudaStream_t s);

cudaError_t launch_append_pages(const AppendPagesArgs& a, int dtype, int n_sms, cudaStream_t s);
cudaError_t launch_read_pages(const ReadPagesArgs& a, int dtype, int n_sms, cudaStream_t s);

enum : int { kErrBadPage = 2 };  // with kErrWaitTimeout, the status bits

#ifdef __CUDACC__
// The sequence whose rows q_start[i] .. q_start[i+1]-1 hold `row`, or -1:
// a 32-way search by the whole warp (two dependent loads for 1024 sequences).
// Of equal starts (empty sequences) the last one wins.
__device__ __forceinline__ int find_seq(const PageBatch& b, int row) {
    const int lane = threadIdx.x & 31;
    int lo = 0, hi = b.n_seqs;
    if (hi <= 0 || b.q_start[0] > row) return -1;
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32;
        const int at = lo + (lane + 1) * step;
        const bool le = at < hi && b.q_start[at] <= row;
        const int n = __popc(__ballot_sync(0xffffffffu, le));
        lo += n * step;
        hi = min(hi, lo + step);
    }
    return row < b.q_start[lo + 1] ? lo : -1;
}

// The page of own position `pos` of sequence i, or -1 when the table or the
// pool does not have it.
__device__ __forceinline__ int page_of(const PagePool& p, const PageBatch& b, int i, int pos) {
    const int j = pos >> 8;
    if (j >= b.table_stride) return -1;
    const int page = b.table[(size_t)i * b.table_stride + j];
    return (unsigned)page < (unsigned)p.n_pages ? page : -1;
}

// The sequence of `row` by one thread's bisection (rows outside the batch: -1).
__device__ __forceinline__ int find_seq_thread(const PageBatch& b, int row) {
    int lo = 0, hi = b.n_seqs;
    if (hi <= 0 || b.q_start[0] > row) return -1;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (b.q_start[mid] <= row) lo = mid; else hi = mid;
    }
    return row < b.q_start[lo + 1] ? lo : -1;
}

// What a row sees: absolute position and keys first <= j < end (absolute).
struct RowView {
    int pos, first, end;
};
__device__ __forceinline__ RowView row_view(const AttendPagesArgs& a, int seq, int row) {
    RowView v;
    const int len = max(a.batch.seq_len[seq], 0);
    // in 64 bits: a length near 2^31 behind a prefix and the largest window before
    // position -1 pass int32 (such a length is beyond any page table and ends as bad)
    const long long pos = (long long)a.prefix_len + a.batch.seq_len[seq] - ((long long)a.batch.q_start[seq + 1] - row);
    v.pos = (int)max(min(pos, 0x7ffffffell), -0x7fffffffll);
    v.first = a.first_key ? a.first_key[row] : (a.window > 0 ? (int)max((long long)v.pos - a.window + 1, 0ll) : 0);
    v.end = a.end_key ? a.end_key[row] : v.pos + 1;
    v.first = max(v.first, 0);
    // 0 .. the keys that exist: callers subtract the prefix from it, which an end far below 0 would not survive
    v.end = max(0, (int)min((long long)v.end, (long long)a.prefix_len + len));
    return v;
}

// 2^x with the hardware approximation (flush-to-zero; 2^-inf = 0)
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// tanh as 1 - 2 / (e^2x + 1): 3 * 2^-23 absolute, so a capped score is off by
// at most 4e-7 of its cap
__device__ __forceinline__ float tanh_abs(float x) {
    return 1.0f - __fdividef(2.0f, exp2_fast(x * 2.8853900817779268f) + 1.0f);
}
// score of one key in the log2 domain from the product q.k times scale
__device__ __forceinline__ float score_log2(const AttendPagesArgs& a, float s, float slope, int pos, int key) {
    if (a.softcap > 0.0f) s = a.softcap * tanh_abs(s * a.inv_cap);
    return (s - slope * fabsf((float)(pos - key))) * 1.4426950408889634f;
}
#endif

}  // namespace kvs
