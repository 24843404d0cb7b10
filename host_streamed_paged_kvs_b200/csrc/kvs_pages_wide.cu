// kvs_pages_wide.cu -- attention of many rows per kv head over quantized pages
// found through page tables, on the tcgen05 tensor cores (kvs_attend_pages:
// prompt chunks, and a prefix that many sequences share).
//
// What bounds it: the tensor cores.  Every (row, key) pair costs 512 flops; 256
// rows against 128 keys are 16.8 MFLOP, 2,050 cycles of an SM at the dense rate
// (2,400 at the rate that N = 128 instructions reach), beside 2,050 cycles of
// exponentials (16 a cycle) and the conversion of 32,768 codes.  Measured: 4,280
// cycles a stage at 1.66 GHz, and about 20,000 a unit beside its stages; 256 query
// tokens at 64K with 40 / 8 heads 429 us, 800 TFLOP/s.
//
// A unit is (row group of 256 rows, kv head): two 128-row tiles that share every
// converted stage of 128 keys.  A planning launch finds each group's stages
// (causal bounds, windows and key intervals cut them) on the device; all units'
// stages form one list and every CTA takes an equal run of it.  Units that
// several CTAs share leave records, which a last launch joins in CTA order.
//
// Roles, handing work over by mbarriers only, 16 warps:
//   warps 0..3, 4..7: softmax of tile 0 and 1, a thread a row.  S comes 64 keys
//     at a time in two buffers of tensor memory, so that the next scores are there
//     when a sub-stage is done; the weights 2^(s - r) with the row's kept reference
//     are packed to fp16 and put back over S.  A row's maximum is taken only when
//     its weights' sum says that the reference is too low (over 2^13, or the first
//     keys seen): then the row of O is rescaled, once the product before is
//     complete.
//   warps 8..11 and 12..14: convert K and V of each stage to fp16 operand tiles
//     (128-byte swizzle); the next stage's codes are on their way to registers
//     meanwhile.  fp16 rows come by TMA instead, as they are.
//   warp 15: its elected lane issues S = Q K^T of both tiles a sub-stage ahead,
//     and O += P V as the weights come.
// K and V are rounded to fp16 once (d q), the weights once; sums and softmax
// statistics are fp32.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math_constants.h>

#include <algorithm>
#include <atomic>
#include <climits>

#include "kvs_pages.h"
#include "kvs_pages_finish.cuh"
#include "kvs_ptx.cuh"

namespace kvs {
namespace {

constexpr int kSoftWarps = 8, kKWarps = 4, kVWarps = 3, kMmaWarp = kSoftWarps + kKWarps + kVWarps;
constexpr int kThreads = (kMmaWarp + 1) * 32;
constexpr int kStageKeys = 128;
constexpr int kTileBytes = 128 * kHeadDim * 2;        // 32 KB: an operand of 128 rows x 128 fp16
constexpr int kBufs = 2;
constexpr int kOffQ = 0;                              // [tile]
constexpr int kOffK = 2 * kTileBytes;                 // [buffer]
constexpr int kOffV = kOffK + kBufs * kTileBytes;
constexpr int kOffBar = kOffV + kBufs * kTileBytes;
constexpr size_t kSmem = 1024 + kOffBar + 256;
static_assert(kSmem <= 232448, "shared memory");
constexpr float kSumMost = 8192.0f;                   // a row's weights of one stage: fp16 holds each
constexpr uint32_t kColS = 0, kColO = 256;            // tensor memory columns, + 128 per tile
constexpr int kSubKeys = 64;                          // keys of an S tile: two per stage
// f16 x f16 -> f32, M = 128, A K-major (Q) or from tensor memory (P); S: N = 64 keys, B K-major; PV: N = 128 dims, B MN-major
constexpr uint32_t kIdescS = (1u << 4) | ((64u >> 3) << 17) | ((128u >> 4) << 24);
constexpr uint32_t kIdescPV = (1u << 4) | (1u << 16) | ((128u >> 3) << 17) | ((128u >> 4) << 24);

// shared-memory matrix descriptor (version 1, 128-byte swizzle): rows of 128
// bytes in groups of 8, 64-column halves 16 KB apart
__device__ __forceinline__ uint64_t smem_desc(uint32_t start, uint32_t lbo, uint32_t sbo) {
    return (uint64_t)((start >> 4) & 0x3FFF) | ((uint64_t)((lbo >> 4) & 0x3FFF) << 16) | ((uint64_t)((sbo >> 4) & 0x3FFF) << 32) |
           (1ull << 46) | (2ull << 61);
}
__device__ __forceinline__ uint64_t desc_k(uint32_t base, int kk) {  // dims 16 kk ..
    return smem_desc(base + (kk >> 2) * 16384 + (kk & 3) * 32, 16, 1024);
}
__device__ __forceinline__ uint64_t desc_mn(uint32_t base, int kk) {  // keys 16 kk ..
    return smem_desc(base + kk * 2048, 16384, 1024);
}
// byte offset of the 16-byte chunk (8 columns) c of a row
__device__ __forceinline__ uint32_t chunk_off(int row, int c) {
    return (uint32_t)((c >> 3) * 16384 + row * 128 + (((c & 7) ^ (row & 7)) << 4));
}

__device__ __forceinline__ __half2 u2h(uint32_t u) { return *reinterpret_cast<__half2*>(&u); }
__device__ __forceinline__ uint32_t h2u(__half2 v) { return *reinterpret_cast<uint32_t*>(&v); }
__device__ __forceinline__ void arrive(uint64_t* bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void tma4(void* dst, const CUtensorMap* map, int c0, int c1, int c2, int c3, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(smem_u32(bar)) : "memory");
}
// Products and commits by the elected lane of a converged warp (`one` is 1 in
// that lane): descriptors stay warp-uniform values, so that an instruction is
// issued in a few cycles.  Inside a one-lane branch each descriptor word is
// moved to a uniform register first, 60 to 150 cycles an instruction beside the
// other warps' arithmetic, which made the issue the kernel's bound.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc, uint32_t one) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc), "r"(one)
        : "memory");
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc, uint32_t one) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"(one)
        : "memory");
}
__device__ __forceinline__ void commit_one(uint64_t* bar, uint32_t one) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)), "r"(one)
        : "memory");
}
__device__ __forceinline__ uint32_t elect_one() {
    uint32_t one;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}" : "=r"(one));
    return one;
}
__device__ __forceinline__ unsigned long long f2_bits(float a, float b) {
    return (unsigned long long)__float_as_uint(a) | ((unsigned long long)__float_as_uint(b) << 32);
}
// packed pairs of fp32: a * b + c, a + b
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    unsigned long long r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(f2_bits(a.x, a.y)), "l"(f2_bits(b.x, b.y)), "l"(f2_bits(c.x, c.y)));
    return make_float2(__uint_as_float((uint32_t)r), __uint_as_float((uint32_t)(r >> 32)));
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    unsigned long long r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(f2_bits(a.x, a.y)), "l"(f2_bits(b.x, b.y)));
    return make_float2(__uint_as_float((uint32_t)r), __uint_as_float((uint32_t)(r >> 32)));
}
// 16 columns into tensor memory, without waiting for them
__device__ __forceinline__ void tmem_put16(uint32_t taddr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
        "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_put_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void st_chunk(uint8_t* tile, int row, int c, uint4 v) {
    *reinterpret_cast<uint4*>(tile + chunk_off(row, c)) = v;
}

// ---- planning: the groups and the stages that their rows need ----
// A unit's length in the list: its stages, then kUnitCost places without one,
// for what a unit costs beside its stages (Q, the end of its rows).  Without them
// a CTA got 14 one-stage units of packed documents while others got one unit of
// 14 stages.  4,096 packed tokens at 0, 2, 3, 4, 5, 6, 8 places: 367, 207, 204,
// 209, 213, 223, 231 us; 64 sequences on a 32K prefix 163, 158, 155, 154, 154, 155,
// 155; 256 tokens at 64K 428 to 438 whatever it is.
constexpr int kUnitCost = 4;
__device__ __forceinline__ long long span_of(const WideUnit& u) { return u.n_stages + kUnitCost; }

constexpr int kPlanThreads = 1024;

// this phase's sequence i: rows (tokens) and keys
__device__ __forceinline__ void phase_seq(const AttendPagesArgs& a, int i, int& first_token, int& tokens, int& n_keys) {
    const PageBatch& b = a.batch;
    if (a.prefix_phase) {
        first_token = 0;
        tokens = max(0, min(b.n_rows, b.q_start[b.n_seqs]));
        n_keys = a.prefix_len;
    } else {
        first_token = b.q_start[i];
        tokens = min(max(0, b.q_start[i + 1] - first_token), b.n_rows);
        if ((long long)tokens * a.group <= a.few_rows) tokens = 0;  // the other kernel's
        n_keys = max(0, b.seq_len[i]);
    }
}

__device__ __forceinline__ long long block_scan(long long v, long long* sums, long long& all) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const long long u = __shfl_up_sync(0xffffffffu, v, off);
        if (lane >= off) v += u;
    }
    __syncthreads();
    if (lane == 31) sums[warp] = v;
    __syncthreads();
    all = 0;
    for (int w = 0; w < kPlanThreads / 32; ++w) {
        if (w < warp) v += sums[w];
        all += sums[w];
    }
    return v;
}

__global__ void __launch_bounds__(kPlanThreads) wide_plan_kernel(const __grid_constant__ AttendPagesArgs a, int max_groups) {
    __shared__ long long sums[32];
    __shared__ int sUpto[kPlanThreads], sTokens[kPlanThreads];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int n_seqs = a.prefix_phase ? 1 : a.batch.n_seqs;
    int n_groups = 0;
    for (int i0 = 0; i0 < n_seqs; i0 += kPlanThreads) {
        const int i = i0 + tid;
        int first_token = 0, tokens = 0, n_keys = 0;
        if (i < n_seqs) phase_seq(a, i, first_token, tokens, n_keys);
        const int mine = (int)(((long long)tokens * a.group + kWideRows - 1) / kWideRows);
        long long all;
        const long long upto = block_scan(mine, sums, all);
        sUpto[tid] = (int)upto;
        sTokens[tid] = tokens;
        __syncthreads();
        // a warp per group
        for (int g = warp; g < (int)all; g += kPlanThreads / 32) {
            int lo = 0, hi = kPlanThreads - 1;  // the first thread whose sum passes g
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                if (sUpto[mid] > g) hi = mid; else lo = mid + 1;
            }
            if (n_groups + g >= max_groups) break;  // a malformed batch whose ranges overlap
            int ft, tk, keys;
            phase_seq(a, i0 + lo, ft, tk, keys);
            const int tk_all = a.prefix_phase ? tk : a.batch.q_start[i0 + lo + 1] - ft;
            const int before = lo > 0 ? sUpto[lo - 1] : 0;
            WideUnit u;
            u.seq = i0 + lo;
            u.row0 = (g - before) * kWideRows;
            u.rows = min(kWideRows, sTokens[lo] * a.group - u.row0);
            u.n_keys = keys;
            u.before = 0;
            const int t0 = ft + u.row0 / a.group, t1 = ft + (u.row0 + u.rows - 1) / a.group;
            const int shift = a.prefix_phase ? 0 : a.prefix_len;
            int from = INT_MAX, to = 0;
            if (!a.first_key && !a.end_key && a.window <= 0) {
                // causal only: the last row sees the most; the prefix is taken whole
                from = 0;
                to = keys;
                if (!a.prefix_phase) to = min(keys, max(0, a.batch.seq_len[u.seq] - (ft + tk_all - 1 - t1)));
            } else
            for (int t = t0 + lane; t <= t1; t += 32) {
                if ((unsigned)t >= (unsigned)a.batch.n_rows) continue;
                const int of = a.prefix_phase ? find_seq_thread(a.batch, t) : u.seq;
                if (of < 0) continue;
                const RowView v = row_view(a, of, t);
                const int f = max(v.first - shift, 0), e = min(v.end - shift, keys);
                if (f < e) {
                    from = min(from, f);
                    to = max(to, e);
                }
            }
#pragma unroll
            for (int off = 16; off; off >>= 1) {
                from = min(from, __shfl_xor_sync(0xffffffffu, from, off));
                to = max(to, __shfl_xor_sync(0xffffffffu, to, off));
            }
            // A group that sees no key has one stage of no keys: none of its page numbers is
            // judged (released pages may stand there), and its values count as 0
            if (from >= to) u.n_keys = 0;
            // keys beyond the page table are nobody's: such a unit comes out as NaN
            if (!a.prefix_phase) to = (int)min((long long)to, (long long)a.batch.table_stride * kPageTokens);
            u.stage0 = from < to ? from / kStageKeys : 0;
            u.n_stages = from < to ? (to + kStageKeys - 1) / kStageKeys - u.stage0 : 1;
            if (lane == 0) a.units[n_groups + g] = u;
        }
        n_groups = min(n_groups + (int)all, max_groups);
        __syncthreads();
    }
    long long total = 0;
    for (int g0 = 0; g0 < n_groups; g0 += kPlanThreads) {
        const int g = g0 + tid;
        const long long n = g < n_groups ? span_of(a.units[g]) : 0;
        long long all;
        const long long upto = block_scan(n, sums, all);
        if (g < n_groups) a.units[g].before = total + upto - n;
        total += all;
    }
    if (tid == 0) {
        a.plan->n_groups = n_groups;
        a.plan->total = total;
    }
}

// A CTA's (or a join's) way through the list.  Position x of the list, n_kv *
// total long, lies in group g with n_kv * before_g <= x.
struct Walk {
    WideUnit u;
    int group, h;             // group and kv head of the current unit
    long long unit0;          // list position of the unit's first stage
    long long unit1, real1;   // of its end, and of the end of its stages
};
__device__ __forceinline__ bool walk_to(const AttendPagesArgs& a, Walk& w, long long x, int n_groups) {
    const int n_kv = a.pool.n_kv;
    while (x >= n_kv * (w.u.before + span_of(w.u))) {
        if (++w.group >= n_groups) return false;
        w.u = a.units[w.group];
    }
    w.h = (int)((x - n_kv * w.u.before) / span_of(w.u));
    w.unit0 = n_kv * w.u.before + w.h * span_of(w.u);
    w.unit1 = w.unit0 + span_of(w.u);
    w.real1 = w.unit0 + w.u.n_stages;
    return true;
}
// The next piece of the run [cur, run1): its first position and stages; cur moves
// past it.  False at the end.
__device__ __forceinline__ bool next_piece(const AttendPagesArgs& a, Walk& w, long long& cur, long long run1, int n_groups, long long& from, int& n_st) {
    while (cur < run1 && walk_to(a, w, cur, n_groups)) {
        from = cur;
        cur = min(run1, w.unit1);
        n_st = (int)(min(cur, w.real1) - from);
        if (n_st > 0) return true;
    }
    return false;
}
// by a whole warp: the group of list position x
__device__ __forceinline__ int find_group(const AttendPagesArgs& a, long long x, int n_groups) {
    const int lane = threadIdx.x & 31;
    int lo = 0, hi = n_groups;
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32, at = lo + (lane + 1) * step;
        const bool le = at < hi && a.pool.n_kv * a.units[at].before <= x;
        const int n = __popc(__ballot_sync(0xffffffffu, le));
        lo += n * step;
        hi = min(hi, lo + step);
    }
    return lo;
}

// one of n_warps producer warps: its loads of a stage, 128-byte rows 4 a load, 64-byte rows 8 a load
__host__ __device__ constexpr int mine128(int n_warps) { return (32 + n_warps - 1) / n_warps; }
__host__ __device__ constexpr int mine64(int n_warps) { return (16 + n_warps - 1) / n_warps; }

// 16 int8 codes times d as two 16-byte chunks
__device__ __forceinline__ void conv_s8(const uint4& c, uint32_t d2, uint4& lo, uint4& hi) {
    const __half2 b = __float2half2_rn(1152.0f), d = u2h(d2);
    auto four = [&](uint32_t w, uint32_t& x, uint32_t& y) {
        w ^= 0x80808080u;
        x = h2u(__hmul2(__hsub2(u2h(__byte_perm(w, 0x64646464u, 0x4140)), b), d));
        y = h2u(__hmul2(__hsub2(u2h(__byte_perm(w, 0x64646464u, 0x4342)), b), d));
    };
    four(c.x, lo.x, lo.y);
    four(c.y, lo.z, lo.w);
    four(c.z, hi.x, hi.y);
    four(c.w, hi.z, hi.w);
}

template <int VT, int KT>
__global__ void __launch_bounds__(kThreads, 1)
    attend_wide_kernel(const __grid_constant__ AttendPagesArgs a, const __grid_constant__ PageMaps maps) {
    using PG = PageGeom<VT, KT>;
    constexpr bool kNibbles = VT != kVF16 && VT != kVQ8_0;  // O's columns: dims 0, 2, 1, 3 of every four
    extern __shared__ uint8_t smem_raw[];
    // aligned by an offset, not through an integer: a pointer made from an integer is
    // a generic one, and every access to it a generic load or store
    uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kOffBar);
    uint64_t* k_full = bars;        // [buffer] K written (a producer warp each; TMA for fp16 K)
    uint64_t* k_free = bars + 2;    // [buffer] every S product that reads it is complete
    uint64_t* v_full = bars + 4;
    uint64_t* v_free = bars + 6;
    uint64_t* v_raw = bars + 8;     // [buffer] fp16 V landed
    uint64_t* s_full = bars + 10;   // [tile][half] S complete
    uint64_t* p_full = bars + 14;   // [tile][half] weights written
    uint64_t* o_done = bars + 18;   // [tile][half] the P V product complete (by half: a waiter is then never
                                    // two phases behind, which would look like none)
    uint64_t* q_full = bars + 22;   // [tile] Q written
    uint64_t* done = bars + 24;     // every product complete
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 25);
    int* sGroup = reinterpret_cast<int*>(tmem_slot + 1);
    volatile int* sAbort = reinterpret_cast<volatile int*>(sGroup + 1);
    int* sSlow = sGroup + 2;        // warps that recompute rows

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int n_kv = a.pool.n_kv;
    if (warp == 0) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    if (tid == 32) {
        *sAbort = 0;
        *sSlow = 0;
        for (int i = 0; i < 2; ++i) {
            mbar_init(&k_full[i], KT == kKF16 ? 1 : kKWarps);
            mbar_init(&k_free[i], 1);
            mbar_init(&v_full[i], kVWarps);
            mbar_init(&v_free[i], 1);
            mbar_init(&v_raw[i], 1);
            mbar_init(&q_full[i], 4);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(&o_done[i], 1);
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], 4);
        }
        mbar_init(done, 1);
        fence_mbar_init();
    }
    const int n_groups = a.plan->n_groups;
    const long long total = a.plan->total * n_kv;
    const long long per = max(1ll, (total + gridDim.x - 1) / gridDim.x);
    const long long run0 = min(total, per * blockIdx.x), run1 = min(total, run0 + per);
    if (warp == 2 && run0 < run1) {
        const int g = find_group(a, run0, n_groups);
        if (lane == 0) *sGroup = g;
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    bool ok = run0 < run1;
    auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {  // by one thread or a whole warp
        if (ok && mbar_try_wait(bar, parity)) return true;
        if (!ok || *sAbort) return ok = false;
        if (!wait_phase(bar, parity, a.batch.status, sSlow)) {
            ok = false;
            *sAbort = 1;
        }
        return ok;
    };
    Walk w;
    w.group = ok ? *sGroup : 0;
    if (ok) w.u = a.units[w.group];
    const int shift = a.prefix_phase ? 0 : a.prefix_len;

    if (warp < kSoftWarps) {
        // ============================ softmax ============================
        const int tile = warp >> 2, trow = (warp & 3) * 32 + lane;  // row of the tile = lane of tensor memory
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t t_s = tmem + lanes + kColS + tile * 128, t_o = tmem + lanes + kColO + tile * 128;
        uint8_t* sq = smem + kOffQ + tile * kTileBytes;
        const bool formed = a.softcap > 0.0f || a.slopes;
        uint32_t n_sub = 0;  // sub-stages of this tile so far: S, P and O phases go by it
        long long cur = run0, from = 0;
        int n_st = 0;
        while (next_piece(a, w, cur, run1, n_groups, from, n_st)) {
            const int st0 = w.u.stage0 + (int)(from - w.unit0);
            const int tiles = w.u.rows > 128 ? 2 : 1;
            if (tile >= tiles) continue;
            // ---- this thread's row ----
            const int r = tile * 128 + trow;
            int token = -1, head = 0, seq = w.u.seq, pos = 0, first = 0, end = 0;
            float sc = 0.0f, slope = 0.0f;
            if (r < w.u.rows) {
                const int ft = a.prefix_phase ? 0 : a.batch.q_start[seq];
                const int fr = w.u.row0 + r;
                token = ft + fr / a.group;
                head = w.h * a.group + fr % a.group;
                if ((unsigned)token >= (unsigned)a.batch.n_rows) token = -1;
                if (token >= 0 && a.prefix_phase) {
                    seq = find_seq_thread(a.batch, token);
                    if (seq < 0) token = -1;
                }
            }
            if (token >= 0) {
                const RowView v = row_view(a, seq, token);
                pos = v.pos - shift;
                first = max(v.first - shift, 0);
                end = min(v.end - shift, w.u.n_keys);
                if (a.slopes) slope = a.slopes[head];
            }
            {
                // Q: fp16 as it is; bf16 with the row's power of two taken out
                const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q.p) + (long long)max(token, 0) * a.q.row +
                                                                  (long long)head * a.q.head);
                uint4 v[16];  // the whole row on its way at once
#pragma unroll
                for (int c = 0; c < 16; ++c) v[c] = token >= 0 ? src[c] : make_uint4(0u, 0u, 0u, 0u);
                float up = 1.0f;
                // a negative scale turns Q, so that the largest product is the largest score
                if (a.q_dtype == kDtBF16) {
                    uint32_t top = 0;  // the largest magnitude's bits
#pragma unroll
                    for (int c = 0; c < 16; ++c) {
                        const uint32_t x[4] = {v[c].x, v[c].y, v[c].z, v[c].w};
#pragma unroll
                        for (int i = 0; i < 4; ++i) top = max(top, max(x[i] & 0x7fffu, (x[i] >> 16) & 0x7fffu));
                    }
                    const uint32_t ex = top >> 7;
                    const bool plain = ex < 2 || ex > 252;  // zero, subnormal and non-finite rows
                    const float sign = a.scale < 0.0f ? -1.0f : 1.0f;
                    const float down = plain ? sign : sign * __uint_as_float((254u - ex) << 23);
                    if (!plain) up = __uint_as_float(ex << 23);
                    auto two = [&](uint32_t x) {
                        return h2u(__floats2half2_rn(__uint_as_float(x << 16) * down, __uint_as_float(x & 0xffff0000u) * down));
                    };
#pragma unroll
                    for (int c = 0; c < 16; ++c) st_chunk(sq, trow, c, make_uint4(two(v[c].x), two(v[c].y), two(v[c].z), two(v[c].w)));
                } else {
                    const uint32_t sign = a.scale < 0.0f ? 0x80008000u : 0u;
#pragma unroll
                    for (int c = 0; c < 16; ++c) st_chunk(sq, trow, c, make_uint4(v[c].x ^ sign, v[c].y ^ sign, v[c].z ^ sign, v[c].w ^ sign));
                }
                sc = fabsf(formed ? a.scale : a.scale * 1.4426950408889634f) * up;
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) arrive(&q_full[tile]);
            // A row that sees a key of a page outside the pool, or beyond the page table,
            // comes out as NaN.  Rarely are there such pages among the piece's: then
            // each row judges those it sees.
            bool bad = false;
            {
                const int* table = a.prefix_phase ? a.prefix_table : a.batch.table + (size_t)w.u.seq * a.batch.table_stride;
                const int n_table = a.prefix_phase ? (a.prefix_len + kPageTokens - 1) / kPageTokens : a.batch.table_stride;
                bool some = !a.prefix_phase && max((long long)first, (long long)n_table * kPageTokens) < end;
                for (int j = (st0 >> 1) + lane; 2 * j < st0 + n_st && j * kPageTokens < w.u.n_keys; j += 32)
                    some |= j >= n_table || (unsigned)table[j] >= (unsigned)a.pool.n_pages;
                if (__any_sync(0xffffffffu, some))
                    bad = sees_bad_page(table, n_table, a.pool.n_pages, first, end, st0 * kStageKeys, (st0 + n_st) * kStageKeys);
            }

            float ref = token >= 0 ? -CUDART_INF_F : 0.0f, l = 0.0f;
            // keys that every row of this warp sees
            const int all_from = __reduce_max_sync(0xffffffffu, token >= 0 ? first : 0);
            const int all_to = __reduce_min_sync(0xffffffffu, token >= 0 ? end : INT_MAX);
            for (int i = 0; i < 2 * n_st; ++i, ++n_sub) {
                const int key0 = st0 * kStageKeys + i * kSubKeys;
                const int hb = n_sub & 1;  // which of the tile's two S buffers
                const uint32_t t_sub = t_s + 64 * hb;
                wait(&s_full[2 * tile + hb], (n_sub >> 1) & 1);
                if (!__all_sync(0xffffffffu, ok)) break;
                tc_fence_after();
                const bool masked = key0 < all_from || key0 + kSubKeys > all_to;  // uniform
                if (formed || masked) {
                    // caps, distances and masks: the scores are formed in place first, so that
                    // the pass below stays short
#pragma unroll 1
                    for (int c0 = 0; c0 < kSubKeys; c0 += 32) {
                        float s[32];
                        tmem_ld32(t_sub + c0, s);
                        if (a.softcap > 0.0f) {
                            const float in = sc * a.inv_cap * 2.8853900817779268f, cap = a.softcap * 1.4426950408889634f;
#pragma unroll
                            for (int c = 0; c < 32; ++c)  // cap tanh(x): cap - 2 cap / (e^2x + 1)
                                s[c] = fmaf(-2.0f * cap, __fdividef(1.0f, exp2_fast(s[c] * in) + 1.0f), cap);
                        }
                        if (a.slopes) {
                            const float k = slope * -1.4426950408889634f, m = a.softcap > 0.0f ? 1.0f : sc * 1.4426950408889634f;
                            const float d = (float)(pos - key0 - c0);
#pragma unroll
                            for (int c = 0; c < 32; ++c) s[c] = fmaf(fabsf(d - (float)c), k, s[c] * m);
                        }
                        if (masked) {
                            const int f = min(max(first - key0 - c0, 0), 32), e = min(max(end - key0 - c0, 0), 32);
                            const uint32_t seen = e > f ? (0xffffffffu >> (32 - e + f)) << f : 0u;  // bits f .. e - 1
#pragma unroll
                            for (int c = 0; c < 32; ++c)
                                if (!((seen >> c) & 1u)) s[c] = -CUDART_INF_F;
                        }
                        tmem_st32(t_sub + c0, s);
                    }
                }
                const float mul = formed ? 1.0f : sc;
                // ---- weights with the row's kept reference; put back over the scores when the
                // row's sum says that the reference stands ----
                const float2 mul2 = make_float2(mul, mul);
                uint32_t p[32];
                float sum;
#pragma unroll 1
                for (int round = 0;; ++round) {
                    const float mu = ref == -CUDART_INF_F ? 0.0f : -ref;
                    const float2 mu2 = make_float2(mu, mu);
                    float2 s0 = make_float2(0.0f, 0.0f), s1 = make_float2(0.0f, 0.0f);
#pragma unroll
                    for (int c0 = 0; c0 < kSubKeys; c0 += 32) {  // 64 at once would not fit the registers
                        float x[32];
                        tmem_ld32(t_sub + c0, x);
#pragma unroll
                        for (int c = 0; c < 32; c += 4) {
                            float2 u = fma2(make_float2(x[c], x[c + 1]), mul2, mu2);
                            float2 v = fma2(make_float2(x[c + 2], x[c + 3]), mul2, mu2);
                            u = make_float2(exp2_fast(u.x), exp2_fast(u.y));
                            v = make_float2(exp2_fast(v.x), exp2_fast(v.y));
                            s0 = add2(s0, u);
                            s1 = add2(s1, v);
                            p[(c0 + c) / 2] = h2u(__floats2half2_rn(u.x, u.y));
                            p[(c0 + c) / 2 + 1] = h2u(__floats2half2_rn(v.x, v.y));
                        }
                    }
                    s0 = add2(s0, s1);
                    sum = s0.x + s0.y;
                    const bool low = token >= 0 && (!(sum <= kSumMost) || (ref == -CUDART_INF_F && max(first, key0) < min(end, key0 + kSubKeys)));
                    if (round || !__any_sync(0xffffffffu, low)) break;
                    // the row's maximum: the reference goes 4 below it, and O with it
                    float top = -CUDART_INF_F;
#pragma unroll 1
                    for (int c0 = 0; c0 < kSubKeys; c0 += 32) {
                        float x[32];
                        tmem_ld32(t_sub + c0, x);
#pragma unroll
                        for (int c = 0; c < 32; ++c) top = fmaxf(top, x[c]);
                    }
                    const float now = low ? fmaxf(ref, top * mul - 4.0f) : ref;
                    const float f = now == ref ? 1.0f : exp2_fast(ref - now);
                    ref = now;
                    l *= f;
                    if (i > 0) {
                        // the product before must be complete; the next one needs this warp's weights
                        wait(&o_done[2 * tile + (hb ^ 1)], ((n_sub - 1) >> 1) & 1);
                        tc_fence_after();
#pragma unroll 1
                        for (int c = 0; c < 128; c += 32) {
                            float o[32];
                            tmem_ld32(t_o + c, o);
#pragma unroll
                            for (int j = 0; j < 32; ++j) o[j] *= f;
                            tmem_st32(t_o + c, o);
                        }
                    }
                }
                if (!__all_sync(0xffffffffu, ok)) break;
                l += sum;
                tmem_put16(t_sub, p);
                tmem_put16(t_sub + 16, p + 16);
                tmem_put_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) arrive(&p_full[2 * tile + hb]);
            }
            if (!__all_sync(0xffffffffu, ok)) break;
            wait(&o_done[2 * tile + 1], ((n_sub - 1) >> 1) & 1);
            if (!__all_sync(0xffffffffu, ok)) break;
            tc_fence_after();

            // ---- the piece's end: O through shared memory (this warp's rows of Q), 64
            // dims at a time, so that rows move as whole lines ----
            const bool whole = w.unit0 >= run0 && w.real1 <= run1;
            if (bad) l = CUDART_NAN_F;
            const int slot = w.unit0 < run0 ? 0 : 1;
            const size_t at = (size_t)max(token, 0) * a.n_qh + head;
            float M = ref, L = l, wo = 1.0f, wp = 0.0f;  // own and prefix weights
            const bool final_rows = whole && !a.prefix_phase;
            if (final_rows) {
                if (a.prefix_len > 0 && token >= 0) {
                    const float2 ml = a.prior_ml[at];
                    M = fmaxf(ref, ml.x);
                    wo = ref == M ? 1.0f : exp2_fast(ref - M);
                    wp = ml.x == M ? 1.0f : exp2_fast(ml.x - M);
                    L = l * wo + ml.y * wp;
                }
                const float inv = L != 0.0f ? 1.0f / L : 0.0f;
                wo *= inv;
                wp *= inv;
                if (token >= 0 && a.lse) a.lse[at] = L == 0.0f ? -CUDART_INF_F : (M + log2f(L)) * 0.69314718055994531f;
            } else if (token >= 0) {
                if (whole) a.prior_ml[at] = make_float2(M, L);
                else {
                    float* rec = a.records + ((size_t)(blockIdx.x * 2 + slot) * kWideRows + r) * kRecordFloats;
                    *reinterpret_cast<float2*>(rec + 128) = make_float2(M, L);
                }
            }
            const bool finite = L * 0.0f == 0.0f;
            uint32_t redo = 0;  // rows of this warp that an unseen value spoiled
            // staging: 32 rows x 256 bytes in the warp's two 4 KB parts, 16-byte chunks turned by the row
            auto stage = [&](int row, int chunk) {
                return reinterpret_cast<float4*>(sq + (row >> 4) * 16384 + (warp & 3) * 4096 + (row & 15) * 256 + ((chunk ^ (row & 15)) << 4));
            };
            // where this thread's row goes, in values (-1: nowhere)
            long long to = -1;
            if (token >= 0)
                to = final_rows ? token * a.out.row + head * a.out.head
                                : (whole ? (long long)at * kHeadDim
                                         : ((long long)(blockIdx.x * 2 + slot) * kWideRows + r) * kRecordFloats);
            float* keep = whole ? a.prior_acc : a.records;
#pragma unroll 1
            for (int hf = 0; hf < 2; ++hf) {
#pragma unroll
                for (int c0 = 0; c0 < 64; c0 += 32) {
                    float o[32];
                    tmem_ld32(t_o + 64 * hf + c0, o);
                    if (c0 == 0) __syncwarp();
#pragma unroll
                    for (int c = 0; c < 8; ++c)
                        *stage(lane, c0 / 4 + c) = kNibbles ? make_float4(o[4 * c], o[4 * c + 2], o[4 * c + 1], o[4 * c + 3])
                                                            : make_float4(o[4 * c], o[4 * c + 1], o[4 * c + 2], o[4 * c + 3]);
                }
                __syncwarp();
                const int c = lane & 15, d = 64 * hf + 4 * c;
                if (!final_rows) {
#pragma unroll 4
                    for (int it = 0; it < 16; ++it) {
                        const int row = 2 * it + (lane >> 4);
                        const long long rt = __shfl_sync(0xffffffffu, to, row);
                        if (rt >= 0) *reinterpret_cast<float4*>(keep + rt + d) = *stage(row, c);
                    }
                    continue;
                }
#pragma unroll 4
                for (int it = 0; it < 16; ++it) {
                    const int row = 2 * it + (lane >> 4);
                    float4 v = *stage(row, c);
                    const long long rt = __shfl_sync(0xffffffffu, to, row);
                    const float fo = __shfl_sync(0xffffffffu, wo, row);
                    // a part without weight (nothing of it is seen) does not count, whatever its sums hold
                    v = fo == 0.0f ? make_float4(0.0f, 0.0f, 0.0f, 0.0f) : make_float4(v.x * fo, v.y * fo, v.z * fo, v.w * fo);
                    if (a.prefix_len > 0) {
                        const float fp = __shfl_sync(0xffffffffu, wp, row);
                        const unsigned long long ra = __shfl_sync(0xffffffffu, (unsigned long long)at, row);
                        if (rt >= 0 && fp != 0.0f) {
                            const float4 pv = *reinterpret_cast<const float4*>(a.prior_acc + ra * kHeadDim + d);
                            v = make_float4(fmaf(pv.x, fp, v.x), fmaf(pv.y, fp, v.y), fmaf(pv.z, fp, v.z), fmaf(pv.w, fp, v.w));
                        }
                    }
                    const bool spoiled = rt >= 0 && !((v.x + v.y + v.z + v.w) * 0.0f == 0.0f);
                    if (rt >= 0) store_out4_at(a, rt + d, v);
                    const uint32_t votes = __ballot_sync(0xffffffffu, spoiled);
                    if (votes & 0xffffu) redo |= 1u << (2 * it);
                    if (votes >> 16) redo |= 2u << (2 * it);
                }
            }
            redo &= __ballot_sync(0xffffffffu, finite && L != 0.0f);
            for (; redo; redo &= redo - 1) {
                const int row = __ffs(redo) - 1;
                const int tk = __shfl_sync(0xffffffffu, token, row), hd = __shfl_sync(0xffffffffu, head, row);
                const int sq_ = __shfl_sync(0xffffffffu, seq, row);
                store_out4(a, tk, hd, 4 * lane, slow_row<VT, KT>(a, sq_, tk, hd, sSlow));
            }
            // any row of the warp: a row that ends beyond the table may be in any lane
            if (__any_sync(0xffffffffu, bad) && lane == 0 && a.batch.status) atomicOr(a.batch.status, kErrBadPage);
            __syncwarp();
        }
    } else if (warp < kMmaWarp) {
        // ============================ producers ============================
        // The codes of the next stage are loaded into registers as soon as this
        // stage's are converted.  Lanes are laid out so that the eight lanes of a
        // 16-byte store phase hit distinct banks of the swizzled tiles:
        //   128-byte rows, 4 a load: lane bits (chunk 0, 1), row 0, chunk 2, row 1;
        //   64-byte rows, 8 a load:  lane bits block 0, (row 0, 1), block 1, row 2.
        const int ch = (lane & 3) + 4 * ((lane >> 3) & 1), rl = ((lane >> 2) & 1) + 2 * (lane >> 4);
        const int bv = (lane & 1) + 2 * ((lane >> 3) & 1), rv = ((lane >> 1) & 3) + 4 * (lane >> 4);
        // the stage after (piece, stage): pieces follow each other without a break
        struct Next {
            const uint8_t* ph;
            int hp, t0, valid;
            bool there;
        };
        long long cur = run0;
        int st = 0, left = 0;
        int pages = 0, pages_at = -1;
        const int* table = nullptr;
        int n_table = 0;
        auto advance = [&]() -> Next {
            Next x{nullptr, 0, 0, 0, false};
            if (left == 0) {  // the next piece
                long long from;
                if (!next_piece(a, w, cur, run1, n_groups, from, left)) return x;
                st = w.u.stage0 + (int)(from - w.unit0);
                table = a.prefix_phase ? a.prefix_table : a.batch.table + (size_t)w.u.seq * a.batch.table_stride;
                n_table = a.prefix_phase ? (a.prefix_len + kPageTokens - 1) / kPageTokens : a.batch.table_stride;
                pages_at = -1;
            }
            const int j = st >> 1;
            if (pages_at < 0 || j >= pages_at + 32) {
                pages_at = j;
                pages = j + lane < n_table ? table[j + lane] : -1;
            }
            int page = __shfl_sync(0xffffffffu, pages, j - pages_at);
            if ((unsigned)page >= (unsigned)a.pool.n_pages) page = 0;  // some page: the softmax warps see it too
            x.hp = page * n_kv + w.h;
            x.ph = a.pool.pages + (size_t)x.hp * PG::kHeadBytes;
            x.t0 = (st & 1) * kStageKeys;
            x.valid = w.u.n_keys - st * kStageKeys;  // tokens of the stage that exist
            x.there = true;
            ++st;
            --left;
            return x;
        };
        if (warp < kSoftWarps + kKWarps) {
            // ---- K ----
            const int pw = warp - kSoftWarps;
            constexpr int kMine = KT == kKF16 ? 1 : mine128(kKWarps);
            uint4 kc[kMine];
            __half kd[kMine];
            auto load_k = [&](const Next& x) {
                if constexpr (KT == kKQ8_0) {
#pragma unroll
                    for (int g = 0; g < kMine; ++g) {
                        const int row = x.t0 + 4 * (pw + kKWarps * g) + rl;
                        if (pw + kKWarps * g < 32) {
                            kc[g] = *reinterpret_cast<const uint4*>(x.ph + row * 128 + 16 * ch);
                            kd[g] = *reinterpret_cast<const __half*>(x.ph + PG::kOffKd + row * 8 + (ch & ~1));
                        }
                    }
                }
            };
            Next x{nullptr, 0, 0, 0, false};
            if (ok) x = advance();
            if (x.there) load_k(x);
            for (uint32_t n = 0; x.there; ++n) {
                const Next y = advance();
                const int kb = n & 1;
                if (n >= 2) {
                    wait(&k_free[kb], ((n >> 1) - 1) & 1);
                    if (!__all_sync(0xffffffffu, ok)) break;
                }
                uint8_t* kt = smem + kOffK + kb * kTileBytes;
                if constexpr (KT == kKQ8_0) {
#pragma unroll
                    for (int g = 0; g < kMine; ++g) {
                        const int row = 4 * (pw + kKWarps * g) + rl;
                        if (pw + kKWarps * g < 32) {
                            uint4 lo, hi;
                            conv_s8(kc[g], h2u(__half2half2(kd[g])), lo, hi);
                            st_chunk(kt, row, 2 * ch, lo);
                            st_chunk(kt, row, 2 * ch + 1, hi);
                        }
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) arrive(&k_full[kb]);
                    if (y.there) load_k(y);
                } else if (pw == 0 && lane == 0) {
                    mbar_expect_tx(&k_full[kb], kTileBytes);
                    tma4(kt, &maps.k, 0, 0, x.t0, x.hp, &k_full[kb]);
                    tma4(kt + 16384, &maps.k, 0, 1, x.t0, x.hp, &k_full[kb]);
                }
                x = y;
            }
        } else {
            // ---- V: rows that do not exist hold anything, their values become 0 ----
            const int pw = warp - kSoftWarps - kKWarps;
            constexpr int kMine = VT == kVF16 ? 1 : (VT == kVQ8_0 ? mine128(kVWarps) : mine64(kVWarps));
            uint4 vc[kMine];
            __half vd[kMine], vm[kMine];
            uint32_t vh[kMine];
            auto load_v = [&](const Next& x) {
                const uint8_t* vq = x.ph + PG::kOffVq;
                if constexpr (VT == kVQ8_0) {
#pragma unroll
                    for (int g = 0; g < kMine; ++g) {
                        const int row = x.t0 + 4 * (pw + kVWarps * g) + rl;
                        if (pw + kVWarps * g < 32) {
                            vc[g] = *reinterpret_cast<const uint4*>(vq + row * 128 + 16 * ch);
                            vd[g] = *reinterpret_cast<const __half*>(x.ph + PG::kOffVd + row * 8 + (ch & ~1));
                        }
                    }
                } else if constexpr (VT != kVF16) {
#pragma unroll
                    for (int g = 0; g < kMine; ++g) {
                        const int row = x.t0 + 8 * (pw + kVWarps * g) + rv;
                        if (pw + kVWarps * g < 16) {
                            vc[g] = *reinterpret_cast<const uint4*>(vq + row * 64 + 16 * bv);
                            vd[g] = *reinterpret_cast<const __half*>(x.ph + PG::kOffVd + row * 8 + 2 * bv);
                            if constexpr (v_has_fifth(VT)) vh[g] = *reinterpret_cast<const uint32_t*>(x.ph + PG::kOffVh + row * 16 + 4 * bv);
                            if constexpr (v_has_min(VT)) vm[g] = *reinterpret_cast<const __half*>(x.ph + PG::kOffVm + row * 8 + 2 * bv);
                        }
                    }
                }
            };
            Next x{nullptr, 0, 0, 0, false};
            if (ok) x = advance();
            if (x.there) load_v(x);
            for (uint32_t n = 0; x.there; ++n) {
                const Next y = advance();
                const int vb = n & 1;
                if (n >= 2) {
                    wait(&v_free[vb], ((n >> 1) - 1) & 1);
                    if (!__all_sync(0xffffffffu, ok)) break;
                }
                uint8_t* vt = smem + kOffV + vb * kTileBytes;
                const __half zero = __float2half(0.0f);
                if constexpr (VT == kVQ8_0) {
#pragma unroll
                    for (int g = 0; g < kMine; ++g) {
                        const int row = 4 * (pw + kVWarps * g) + rl;
                        if (pw + kVWarps * g < 32) {
                            uint4 lo, hi;
                            conv_s8(vc[g], h2u(__half2half2(row < x.valid ? vd[g] : zero)), lo, hi);
                            st_chunk(vt, row, 2 * ch, lo);
                            st_chunk(vt, row, 2 * ch + 1, hi);
                        }
                    }
                } else if constexpr (VT == kVF16) {
                    if (pw == 0 && lane == 0) {
                        mbar_expect_tx(&v_raw[vb], kTileBytes);
                        tma4(vt, &maps.v, 0, 0, PG::kOffVq / 256 + x.t0, x.hp, &v_raw[vb]);
                        tma4(vt + 16384, &maps.v, 0, 1, PG::kOffVq / 256 + x.t0, x.hp, &v_raw[vb]);
                    }
                    wait(&v_raw[vb], (n >> 1) & 1);
                    if (!__all_sync(0xffffffffu, ok)) break;
                    for (int c = pw * 32 + lane; x.valid < kStageKeys && c < 128 * 16; c += kVWarps * 32)
                        if ((c >> 4) >= x.valid) st_chunk(vt, c >> 4, c & 15, make_uint4(0u, 0u, 0u, 0u));
                } else {
#pragma unroll
                    for (int g = 0; g < kMine; ++g) {
                        const int row = 8 * (pw + kVWarps * g) + rv;
                        if (pw + kVWarps * g < 16) {
                            const bool there = row < x.valid;
                            const __half2 d = __half2half2(there ? vd[g] : zero);
                            const __half2 m = v_has_min(VT) ? __half2half2(there ? vm[g] : zero) : __float2half2_rn(0.0f);
                            constexpr float kZero = v_has_min(VT) ? 0.0f : (VT == kVQ5_0 ? 16.0f : 8.0f);
                            const __half2 z = __float2half2_rn(1024.0f + kZero), z16 = __float2half2_rn(-64.0f - kZero);
                            const __half2 sixteenth = __float2half2_rn(0.0625f);
                            const uint32_t words[4] = {vc[g].x, vc[g].y, vc[g].z, vc[g].w};
                            // dims 0..15 (low nibbles), 16..31 (high); of four dims the pairs are (0, 2) and
                            // (1, 3), two masks instead of byte moves: O's columns come out in that order
                            uint32_t o[2][8];
#pragma unroll
                            for (int k = 0; k < 4; ++k)
#pragma unroll
                                for (int e = 0; e < 2; ++e) {
                                    const uint32_t wd = e ? words[k] >> 8 : words[k];
                                    uint32_t lo = (wd & 0x000f000fu) | 0x64006400u, hi = (wd & 0x00f000f0u) | 0x64006400u;
                                    if constexpr (v_has_fifth(VT)) {
                                        const uint32_t b = vh[g] >> (4 * k + e);  // bits 0, 2 and 16, 18
                                        lo |= (b & 1u) << 4 | (b & 4u) << 18;
                                        hi |= (b & 0x10000u) >> 8 | (b & 0x40000u) << 6;
                                    }
                                    const __half2 ql = __hsub2(u2h(lo), z), qh = __hfma2(u2h(hi), sixteenth, z16);
                                    o[0][2 * k + e] = h2u(v_has_min(VT) ? __hfma2(ql, d, m) : __hmul2(ql, d));
                                    o[1][2 * k + e] = h2u(v_has_min(VT) ? __hfma2(qh, d, m) : __hmul2(qh, d));
                                }
#pragma unroll
                            for (int c = 0; c < 4; ++c)
                                st_chunk(vt, row, 4 * bv + c, make_uint4(o[c >> 1][4 * (c & 1)], o[c >> 1][4 * (c & 1) + 1],
                                                                         o[c >> 1][4 * (c & 1) + 2], o[c >> 1][4 * (c & 1) + 3]));
                        }
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) arrive(&v_full[vb]);
                if (y.there) load_v(y);
                x = y;
            }
        }
    } else {
        // ============================ products ============================
        const uint32_t one = elect_one();
        // descriptors of the first operands; the others differ by constants (the address
        // field counts 16 bytes, and 227 KB stay below its 14 bits)
        const uint32_t smem0 = smem_u32(smem);
        const uint64_t dq = desc_k(smem0 + kOffQ, 0), dk = desc_k(smem0 + kOffK, 0), dv = desc_mn(smem0 + kOffV, 0);
        uint32_t n_k = 0, n_v = 0, n_p[2] = {0, 0}, n_q[2] = {0, 0};
        long long cur = run0, from = 0;
        int n_st = 0;
        while (ok && next_piece(a, w, cur, run1, n_groups, from, n_st)) {
            const int tiles = w.u.rows > 128 ? 2 : 1;
            // S of a sub-stage of tile t: 64 keys, half of the stage's K tile
            auto scores = [&](int t, uint32_t half) {
                const uint64_t k = dk + ((n_k & 1) * kTileBytes + half * (kSubKeys * 128)) / 16;
#pragma unroll
                for (int kk = 0; kk < 8; ++kk) {
                    const uint32_t off = ((kk >> 2) * 16384 + (kk & 3) * 32) / 16;
                    mma_ss(tmem + kColS + 128 * t + 64 * half, dq + t * (kTileBytes / 16) + off, k + off, kIdescS, kk > 0, one);
                }
                commit_one(&s_full[2 * t + half], one);
            };
            wait(&k_full[n_k & 1], (n_k >> 1) & 1);
            wait(&q_full[0], n_q[0]++ & 1);
            if (tiles > 1) wait(&q_full[1], n_q[1]++ & 1);
            if (!ok) break;
            tc_fence_after();
            scores(0, 0);
            if (tiles > 1) scores(1, 0);
#pragma unroll 1
            for (int i = 0; i < n_st; ++i) {
#pragma unroll
                for (uint32_t half = 0; half < 2; ++half) {
                    const bool next = half == 0 || i + 1 < n_st;
                    if (half == 1 && next) wait(&k_full[n_k & 1], (n_k >> 1) & 1);
                    if (half == 0) wait(&v_full[n_v & 1], (n_v >> 1) & 1);
                    const uint64_t v = dv + ((n_v & 1) * kTileBytes + half * 4 * 2048) / 16;
                    // a tile's next S goes before its product: the buffer's weights were taken
                    // by the product before, issued already.  Tile by tile, so that the two
                    // tiles' softmax warps do not all work at once
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        if (t >= tiles) break;
                        tc_fence_after();
                        if (next) scores(t, half ^ 1);
                        wait(&p_full[2 * t + half], n_p[t] & 1);  // n_p: stages of this tile
                        tc_fence_after();
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            mma_ts(tmem + kColO + 128 * t, tmem + kColS + 128 * t + 64 * half + 8 * kk, v + kk * (2048 / 16), kIdescPV,
                                   (half || kk) ? 1u : (i > 0), one);
                        commit_one(&o_done[2 * t + half], one);
                    }
                    if (half == 0) {
                        commit_one(&k_free[n_k & 1], one);
                        ++n_k;
                    }
                }
                if (!ok) break;
                commit_one(&v_free[n_v & 1], one);
                ++n_v;
                ++n_p[0];
                if (tiles > 1) ++n_p[1];
            }
        }
        if (run0 < run1) {  // nothing is in flight when the memory is given back
            commit_one(done, one);
            wait_phase(done, 0, a.batch.status, sSlow);
        }
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ---- the join of units that several CTAs share: block (CTA border, rows); the
// border that is the first inside its unit does it, a warp a row ----
constexpr int kJoinWarps = 8;
template <int VT, int KT>
__global__ void __launch_bounds__(kJoinWarps * 32) wide_join_kernel(const __grid_constant__ AttendPagesArgs a, int n_ctas) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int n_groups = a.plan->n_groups;
    const long long total = a.plan->total * a.pool.n_kv, per = max(1ll, (total + n_ctas - 1) / n_ctas);
    const long long x = per * (blockIdx.x + 1);  // the border before CTA blockIdx.x + 1
    if (x >= total) return;
    Walk w;
    w.group = find_group(a, x, n_groups);
    w.u = a.units[w.group];
    // between units or behind a unit's stages, or not the unit's first border
    if (!walk_to(a, w, x, n_groups) || w.unit0 == x || x >= w.real1 || w.unit0 < x - per) return;
    const int c0 = blockIdx.x, c1 = (int)((w.real1 - 1) / per);
    const int ft = a.prefix_phase ? 0 : a.batch.q_start[w.u.seq];
    for (int r = blockIdx.y * kJoinWarps + warp; r < w.u.rows; r += gridDim.y * kJoinWarps) {
        const int fr = w.u.row0 + r, token = ft + fr / a.group, head = w.h * a.group + fr % a.group;
        if ((unsigned)token >= (unsigned)a.batch.n_rows || (a.prefix_phase && find_seq_thread(a.batch, token) < 0)) continue;
        float M = -CUDART_INF_F, L = 0.0f;
        float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        constexpr int kBatch = 8;  // records on their way at once
#pragma unroll 1
        for (int c = c0; c <= c1; c += kBatch) {
            float4 v[kBatch];
            float2 ml[kBatch];
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                const float* rec = a.records + ((size_t)(min(c + b, c1) * 2 + (c + b == c0 ? 1 : 0)) * kWideRows + r) * kRecordFloats;
                v[b] = reinterpret_cast<const float4*>(rec)[lane];
                ml[b] = *reinterpret_cast<const float2*>(rec + 128);
            }
#pragma unroll
            for (int b = 0; b < kBatch; ++b)
                if (c + b <= c1) join(acc, M, L, v[b], ml[b].x, ml[b].y);
        }
        finish_row<VT, KT>(a, w.u.seq, token, head, acc, M, L);
    }
}

template <int VT, int KT>
cudaError_t launch(const AttendPagesArgs& a, const PageMaps& maps, int n_sms, cudaStream_t s) {
    static std::atomic<unsigned long long> configured{0};  // the shared-memory opt-in is per device
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev >= 64 || !(configured.load(std::memory_order_acquire) & (1ull << dev))) {
        const cudaError_t e = cudaFuncSetAttribute(attend_wide_kernel<VT, KT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
        if (e != cudaSuccess) return e;
        if (dev < 64) configured.fetch_or(1ull << dev, std::memory_order_acq_rel);
    }
    const int ctas = std::min(kWideCtas, n_sms);
    const long long groups = wide_groups(a.batch.n_rows, a.group, a.prefix_phase ? 1 : a.batch.n_seqs);
    wide_plan_kernel<<<1, kPlanThreads, 0, s>>>(a, (int)std::min(groups, 0x7fffffffll));
    attend_wide_kernel<VT, KT><<<ctas, kThreads, kSmem, s>>>(a, maps);
    if (ctas > 1) wide_join_kernel<VT, KT><<<dim3(ctas - 1, 16), kJoinWarps * 32, 0, s>>>(a, ctas);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attend_wide(const AttendPagesArgs& a, const PageMaps& maps, int n_sms, cudaStream_t s) {
    if (a.pool.k_type == kKF16) return launch<kVF16, kKF16>(a, maps, n_sms, s);
    switch (a.pool.v_type) {
        case kVF16: return launch<kVF16, kKQ8_0>(a, maps, n_sms, s);
        case kVQ4_1: return launch<kVQ4_1, kKQ8_0>(a, maps, n_sms, s);
        case kVQ5_0: return launch<kVQ5_0, kKQ8_0>(a, maps, n_sms, s);
        case kVQ5_1: return launch<kVQ5_1, kKQ8_0>(a, maps, n_sms, s);
        case kVQ8_0: return launch<kVQ8_0, kKQ8_0>(a, maps, n_sms, s);
        default: return launch<kVQ4_0, kKQ8_0>(a, maps, n_sms, s);
    }
}

}  // namespace kvs
