// kvs_pages_few.cu -- attention of few rows per kv head over quantized pages
// found through page tables (kvs_attend_pages: decode and verify steps, and a
// shared prefix seen by few rows).
//
//   out = sum_j p_j v_j / sum_j p_j,  p_j = 2^(s_j - r),  s_j = log2(e) score(q.k_j)
//
// What bounds it: HBM.  A key costs 208 B per kv head (K Q8_0 / V Q4_0) and is
// read once for all rows of its kv head; at 6.5 TB/s an SM has 9 cycles per
// key for everything else, and the math below takes 23 warp instructions.
// Measured: one 256K sequence with 40 / 8 heads 98 us, 4.4 TB/s (the copies
// alone 84 us); 64 sequences of up to 8K, 32 / 8 heads, 122 us, 3.7 TB/s; one 4K
// sequence 12 us, all of it latency.
//
// Work split.  A unit is (sequence, kv head, up to 8 NT rows); its keys come
// in stages of 128.  All units' stages form one list, and every CTA (two per
// SM where the stages fit) takes an equal run of it, whatever the sequences'
// lengths: one long sequence spreads over all SMs, and many short ones leave
// none idle.  Each CTA finds its run from the lengths in device memory itself
// (a block scan), so there is no planning launch, and a captured graph follows
// the lengths.  A unit that several CTAs share leaves one record per CTA, and
// the CTA that arrives last joins them in CTA order (a fixed order: results do
// not depend on which one that is).
//
// A planning warp walks the run some pieces ahead (a piece is a unit's part in
// this CTA): it puts each one's stages, first page numbers, row bounds and Q
// into shared memory.  A loading warp keeps the stages' TMA copies in flight
// across the pieces' borders.  K rows land with the 128-byte swizzle, 4- and 5-bit V rows
// with the 64-byte swizzle, so that ldmatrix reads eight rows without bank
// conflicts.  Four consumer warps take 32 keys of each stage, with a softmax
// state of their own, and join at the piece's end.
//
// Both products keep the keys and dims on the 16-row side of mma.sync
// m16n8k16 and the query rows on the 8-column side, so no tile row is wasted
// on a step's few rows, and a converted operand serves all NT column tiles:
//   S^T [keys x rows] = K [keys x dims] Q^T: int8 codes are exact in fp16; the
//     fp32 sum of each 32-dim block is multiplied by the key's block scale;
//   O^T [dims x rows] += V^T [dims x keys] P^T: ldmatrix.trans gives a lane the
//     codes of two neighbouring keys in one word, which is the operand's pair;
//     codes are exact, and the weight p d_v (one product in fp16, relative to a
//     reference 2^6 below the maximum so that small weights stay normal) is
//     the other operand, turned by movmatrix.  In precise mode its rounding
//     error goes in as a second term, and the sums are fp32-exact.  Q4_1 and
//     Q5_1 values d q + m are rounded to fp16 instead (weights p).
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

constexpr int kConsumers = 4;
constexpr int kThreads = (kConsumers + 2) * 32;
constexpr int kStageKeys = 128;
constexpr int kLeastStages = 1;                    // a CTA's run
constexpr int kQRow = 288;                         // bytes of a Q row in shared memory: 32 mod 128, so that 4 rows x 32 B are distinct banks
constexpr int kRedRow = 132;                       // floats of a row in the join buffer
constexpr int kRedBytes = kConsumers * 8 * kRedRow * 4;

// A piece: rows of one unit and the stages of it that this CTA takes.
template <int ROWS>
struct Piece {
    int n_stages;             // < 0: no more pieces
    int first_stage;          // of the unit's pages
    int rows, seq, kv_head;
    int full_from, full_to;   // keys every row sees
    int n_keys;               // keys that exist
    int slot;                 // record slot, or -1: the whole unit is here
    int cta0, n_ctas;         // CTAs that share the unit
    uint32_t nan_rows;        // rows that see a page outside the pool, or a key beyond the table, a bit each
    int pages[32];            // the first pages, from first_stage / 2 on
    int token[ROWS], head[ROWS];
    int pos[ROWS], first[ROWS], end[ROWS];  // in keys of this phase
    float scale[ROWS], slope[ROWS];
    alignas(16) uint8_t q[ROWS * kQRow];
};

template <int VT, int KT, int NT>
struct Geo {
    using PG = PageGeom<VT, KT>;
    static constexpr int kRows = 8 * NT;
    static constexpr int kOffV = kStageKeys * PG::kKqRow;
    static constexpr int kOffKd = kOffV + kStageKeys * PG::kVqRow;
    static constexpr int kOffVh = kOffKd + kStageKeys * PG::kKdRow;
    static constexpr int kOffVd = kOffVh + kStageKeys * PG::kVhRow;
    static constexpr int kOffVm = kOffVd + kStageKeys * PG::kVdRow;
    static constexpr int kBytes = kOffVm + kStageKeys * PG::kVmRow;
    static constexpr int kSlots = NT == 1 ? 4 : 3;                // pieces planned ahead
    static constexpr size_t kFixed = 1024 + kRedBytes + kSlots * sizeof(Piece<kRows>) + 512;
    static constexpr int kPerSm = 2 * (2 * (size_t)kBytes + kFixed + 1024) <= 233472 ? 2 : 1;
    static constexpr int kFit = (int)((233472 / kPerSm - 1024 - kFixed) / kBytes);
    static constexpr int kStages = kFit < 4 ? kFit : 4;
    static constexpr size_t kOffRed = (size_t)kStages * kBytes;
    static constexpr size_t kOffPiece = kOffRed + kRedBytes;
    static constexpr size_t kOffBar = kOffPiece + kSlots * sizeof(Piece<kRows>);
    static constexpr size_t kSmem = 1024 + kOffBar + 512;
    static_assert(kBytes % 1024 == 0 && kOffV % 1024 == 0, "swizzled tiles need aligned stages");
    static_assert(kStages >= 2 && kSmem <= 232448 && sizeof(Piece<kRows>) % 16 == 0, "shared memory");
};

__device__ __forceinline__ __half2 u2h(uint32_t u) { return *reinterpret_cast<__half2*>(&u); }
__device__ __forceinline__ uint32_t h2u(__half2 v) { return *reinterpret_cast<uint32_t*>(&v); }

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ uint32_t movm(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void arrive(uint64_t* bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void tma3(void* dst, const CUtensorMap* map, int c0, int c1, int c2, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void tma4(void* dst, const CUtensorMap* map, int c0, int c1, int c2, int c3, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(smem_u32(bar)) : "memory");
}

// four int8 codes (biased by 128) as two fp16 pairs: bytes 0, 1 and 2, 3
__device__ __forceinline__ void s8x4(uint32_t w, uint32_t sel0, uint32_t sel1, uint32_t& lo, uint32_t& hi) {
    const uint32_t x = w ^ 0x80808080u;
    const __half2 b = __float2half2_rn(1152.0f);  // 1024 of the exponent trick + 128 of the bias
    lo = h2u(__hsub2(u2h(__byte_perm(x, 0x64646464u, sel0)), b));
    hi = h2u(__hsub2(u2h(__byte_perm(x, 0x64646464u, sel1)), b));
}

// the batch's work as this phase sees it
struct Seq {
    int row0, rows;           // first row; rows (tokens)
    int n_keys;               // keys that exist
    int stage0;               // first stage any row sees
    int n_groups;             // row groups
    long long n_stages;       // stages per unit, at least 1
};
template <int ROWS>
__device__ __forceinline__ Seq seq_of(const AttendPagesArgs& a, int i) {
    Seq s;
    const PageBatch& b = a.batch;
    int keys;
    if (a.prefix_phase) {
        s.row0 = 0;
        s.rows = max(0, min(b.n_rows, b.q_start[b.n_seqs]));
        keys = a.prefix_len;
        s.n_keys = keys;
        s.stage0 = 0;
    } else {
        s.row0 = b.q_start[i];
        s.rows = min(max(0, b.q_start[i + 1] - s.row0), b.n_rows);
        if ((long long)s.rows * a.group > a.few_rows) s.rows = 0;  // the many-row kernel's
        const long long most = (long long)b.table_stride * kPageTokens;
        s.n_keys = max(0, b.seq_len[i]);
        keys = (int)min((long long)s.n_keys, most);
        s.stage0 = 0;
        if (a.window > 0 && !a.first_key)  // own keys before the first row's window are nobody's
            s.stage0 = (int)max(0ll, min((long long)s.n_keys - s.rows - a.window + 1, (long long)keys - 1)) / kStageKeys;
    }
    s.n_groups = (int)(((long long)s.rows * a.group + ROWS - 1) / ROWS);
    s.n_stages = max(1, (keys + kStageKeys - 1) / kStageKeys - s.stage0);
    return s;
}

// a / b for a >= 0, b > 0: 32-bit where both fit
__device__ __forceinline__ long long quot(long long a, long long b) {
    return ((a | b) >> 32) == 0 ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
}

// PRECISE: the weights' rounding errors go in as a second term (a template
// argument: the branches would keep the compiler from overlapping the blocks)
template <int VT, int KT, int NT, bool PRECISE>
__global__ void __launch_bounds__(kThreads, Geo<VT, KT, NT>::kPerSm)
    attend_few_kernel(const __grid_constant__ AttendPagesArgs a, const __grid_constant__ PageMaps maps) {
    using G = Geo<VT, KT, NT>;
    using PG = PageGeom<VT, KT>;
    constexpr int ROWS = G::kRows, kStages = G::kStages, kSlots = G::kSlots;
    extern __shared__ uint8_t smem_raw[];
    // aligned by an offset, not through an integer: a pointer made from an integer is
    // a generic one, and every access to it a generic load or store
    uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    float* red = reinterpret_cast<float*>(smem + G::kOffRed);
    Piece<ROWS>* pieces = reinterpret_cast<Piece<ROWS>*>(smem + G::kOffPiece);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + G::kOffBar);  // [stage] bytes landed
    uint64_t* empty = full + kStages;                                 // [stage] consumers done
    uint64_t* p_meta = empty + kStages;                               // [piece slot] stages and pages are there
    uint64_t* p_full = p_meta + kSlots;                               // [piece slot] rows and Q too
    uint64_t* p_empty = p_full + kSlots;                              // [piece slot] consumers and loader done
    int* sLast = reinterpret_cast<int*>(p_empty + kSlots);            // this CTA joins the unit
    int* sSlow = sLast + 1;                                           // warps that recompute a row
    float* sml = reinterpret_cast<float*>(p_empty + kSlots + 2);      // [warp][8][2] (reference, sum)

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int n_kv = a.pool.n_kv;
    const int n_seqs = a.prefix_phase ? 1 : a.batch.n_seqs;

    if (tid == 0) {
        *sSlow = 0;
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], kConsumers);
        }
        for (int s = 0; s < kSlots; ++s) {
            mbar_init(&p_meta[s], 1);
            mbar_init(&p_full[s], 1);
            mbar_init(&p_empty[s], kConsumers + 1);
        }
        fence_mbar_init();
    }
    __syncthreads();

    if (warp == kConsumers) {
        // ============================ planner ============================
        // ---- this CTA's run of the list of all units' stages: the sequences' shares,
        // 32 at a time, summed once for the whole and once up to the run's start ----
        auto share = [&](int i) -> long long {
            if (i >= n_seqs) return 0;
            const Seq s = seq_of<ROWS>(a, i);
            return s.n_stages * s.n_groups * n_kv;
        };
        const long long mine = share(lane);  // of the first 32, which are all of most batches
        long long total = mine;
#pragma unroll 4
        for (int i = 32 + lane; i < n_seqs; i += 32) total += share(i);
#pragma unroll
        for (int off = 16; off; off >>= 1) total += __shfl_xor_sync(0xffffffffu, total, off);
        const long long per = max((long long)kLeastStages, quot(total + gridDim.x - 1, gridDim.x));
        const long long run0 = min(total, per * blockIdx.x), run1 = min(total, run0 + per);
        int seq = n_seqs;
        long long base = 0;
        for (int i0 = 0; i0 < n_seqs && run0 < run1; i0 += 32) {
            const long long own = i0 == 0 ? mine : share(i0 + lane);
            long long upto = own;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const long long v = __shfl_up_sync(0xffffffffu, upto, off);
                if (lane >= off) upto += v;
            }
            upto += base;
            const uint32_t past = __ballot_sync(0xffffffffu, upto > run0);
            if (past) {  // the first sequence whose shares pass the run's start
                const int at = __ffs(past) - 1;
                seq = i0 + at;
                base = __shfl_sync(0xffffffffu, upto - own, at);
                break;
            }
            base = __shfl_sync(0xffffffffu, upto, 31);
        }
        long long cur = run0;
        int slot = 0;
        uint32_t slot_phase = 1;  // an unused slot's barrier counts as complete in phase 1
        bool ok = true;
        Seq s = seq < n_seqs ? seq_of<ROWS>(a, seq) : Seq{};
        while (ok) {
            while (seq < n_seqs && cur < run1 && cur >= base + s.n_stages * s.n_groups * n_kv) {
                base += s.n_stages * s.n_groups * n_kv;
                ++seq;
                if (seq < n_seqs) s = seq_of<ROWS>(a, seq);
            }
            Piece<ROWS>& p = pieces[slot];
            ok = __all_sync(0xffffffffu, wait_phase(&p_empty[slot], slot_phase, a.batch.status, sSlow));
            if (!ok || cur >= run1 || seq >= n_seqs) {
                if (lane == 0) p.n_stages = -1;
                __syncwarp();
                if (lane == 0) {
                    arrive(&p_meta[slot]);
                    arrive(&p_full[slot]);
                }
                break;
            }
            const long long unit = quot(cur - base, s.n_stages);
            const long long unit0 = base + unit * s.n_stages, unit1 = unit0 + s.n_stages;
            const long long stop = min(run1, unit1);
            const int group = (int)quot(unit, n_kv), h = (int)(unit - (long long)group * n_kv);
            const int rows = min(ROWS, s.rows * a.group - group * ROWS);
            // bounds of the rows, one lane each
            int first = INT_MAX, end = 0, pos = 0, token = -1, head = 0;
            float slope = 0.0f;
            if (lane < rows) {
                const int r = group * ROWS + lane;
                token = s.row0 + r / a.group;
                head = h * a.group + r % a.group;
                int of = seq;
                if ((unsigned)token >= (unsigned)a.batch.n_rows) token = -1;
                else if (a.prefix_phase) {
                    of = find_seq_thread(a.batch, token);
                    if (of < 0) token = -1;
                }
                if (token >= 0) {
                    const RowView v = row_view(a, of, token);
                    const int shift = a.prefix_phase ? 0 : a.prefix_len;
                    pos = v.pos - shift;
                    first = max(v.first - shift, 0);
                    end = min(v.end - shift, s.n_keys);
                    if (a.slopes) slope = a.slopes[head];
                }
            }
            const bool sees = first < end;
            int lo = sees ? first : INT_MAX, hi = sees ? end : 0;
            int full_from = token >= 0 ? first : 0, full_to = token >= 0 ? end : INT_MAX;
#pragma unroll
            for (int off = 16; off; off >>= 1) {
                lo = min(lo, __shfl_xor_sync(0xffffffffu, lo, off));
                hi = max(hi, __shfl_xor_sync(0xffffffffu, hi, off));
                full_from = max(full_from, __shfl_xor_sync(0xffffffffu, full_from, off));
                full_to = min(full_to, __shfl_xor_sync(0xffffffffu, full_to, off));
            }
            int st0 = s.stage0 + (int)(cur - unit0), st1 = s.stage0 + (int)(stop - unit0);
            if (lo < hi) {
                st0 = max(st0, lo / kStageKeys);
                st1 = min(st1, (hi - 1) / kStageKeys + 1);
            } else st1 = st0;
            if (lane < ROWS) {
                p.token[lane] = token;
                p.head[lane] = head;
                p.pos[lane] = pos;
                p.first[lane] = first;
                p.end[lane] = end;
                p.slope[lane] = slope;
            }
            if (lane == 0) {
                p.n_stages = max(0, st1 - st0);
                p.first_stage = st0;
                p.rows = rows;
                p.seq = seq;
                p.kv_head = h;
                p.full_from = full_from;
                p.full_to = full_to;
                p.n_keys = s.n_keys;
            }
            // the first pages' numbers
            const int* table = a.prefix_phase ? a.prefix_table : a.batch.table + (size_t)seq * a.batch.table_stride;
            const int n_table = a.prefix_phase ? (a.prefix_len + kPageTokens - 1) / kPageTokens : a.batch.table_stride;
            const int j = (st0 >> 1) + lane;
            const int page = 2 * j < st1 && j < n_table ? table[j] : -1;
            p.pages[lane] = page;
            __syncwarp();
            if (lane == 0) arrive(&p_meta[slot]);
            // Where the piece's pages hold a bad number, or a row ends beyond the table, each
            // row judges the keys that it sees
            bool some = max((long long)first, (long long)n_table * kPageTokens) < end || (2 * j < st1 && (unsigned)page >= (unsigned)a.pool.n_pages);
            for (int i = j + 32; 2 * i < st1; i += 32) some |= i >= n_table || (unsigned)table[i] >= (unsigned)a.pool.n_pages;
            uint32_t nan_rows = 0;
            if (__any_sync(0xffffffffu, some)) {
                nan_rows = __ballot_sync(0xffffffffu, sees_bad_page(table, n_table, a.pool.n_pages, first, end, st0 * kStageKeys, st1 * kStageKeys));
                if (nan_rows && lane == 0 && a.batch.status) atomicOr(a.batch.status, kErrBadPage);
            }
            if (lane == 0) p.nan_rows = nan_rows;
            if (lane == 0) {
                // the record slot, and the CTAs that share the unit
                p.slot = (unit0 >= run0 && unit1 <= run1) ? -1 : (unit0 < run0 ? 0 : 1);
                p.cta0 = unit0 >= run0 ? (int)blockIdx.x : (int)quot(unit0, per);
                p.n_ctas = (unit1 <= run1 ? (int)blockIdx.x : (int)quot(unit1 - 1, per)) - p.cta0 + 1;
            }
            // Q: fp16 as it is; bf16 as fp16 after taking each row's power of two
            // out (exact down to 2^-24 of the row's largest value)
            const float unit_scale = a.softcap > 0.0f || a.slopes ? a.scale : a.scale * 1.4426950408889634f;
#pragma unroll 1
            for (int r0 = 0; r0 < ROWS; r0 += 8) {
                uint2 w[8];  // eight rows on their way at once
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const int tk = __shfl_sync(0xffffffffu, token, r0 + k), hd = __shfl_sync(0xffffffffu, head, r0 + k);
                    w[k] = make_uint2(0u, 0u);
                    if (tk >= 0)
                        w[k] = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(a.q.p) + tk * a.q.row + hd * a.q.head + 4 * lane);
                }
                float up[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) up[k] = 1.0f;
                if (a.q_dtype == kDtBF16) {
                    uint32_t top[8];  // the largest magnitude's bits
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        top[k] = max(max(w[k].x & 0x7fffu, (w[k].x >> 16) & 0x7fffu), max(w[k].y & 0x7fffu, (w[k].y >> 16) & 0x7fffu));
#pragma unroll
                    for (int k = 0; k < 8; ++k) top[k] = __reduce_max_sync(0xffffffffu, top[k]);
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        // 2^e with 2^e <= top < 2^(e+1); 1 for zero, subnormal and non-finite rows
                        const uint32_t ex = top[k] >> 7;
                        const bool plain = ex < 2 || ex > 252;
                        const float down = plain ? 1.0f : __uint_as_float((254u - ex) << 23);
                        if (!plain) up[k] = __uint_as_float(ex << 23);
                        *reinterpret_cast<__half2*>(&w[k].x) =
                            __floats2half2_rn(__uint_as_float(w[k].x << 16) * down, __uint_as_float(w[k].x & 0xffff0000u) * down);
                        *reinterpret_cast<__half2*>(&w[k].y) =
                            __floats2half2_rn(__uint_as_float(w[k].y << 16) * down, __uint_as_float(w[k].y & 0xffff0000u) * down);
                    }
                }
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    *reinterpret_cast<uint2*>(p.q + (r0 + k) * kQRow + 8 * lane) = w[k];
                    if (lane == 0) p.scale[r0 + k] = unit_scale * up[k];
                }
            }
            __syncwarp();
            if (lane == 0) arrive(&p_full[slot]);
            cur = stop;
            if (++slot == kSlots) {
                slot = 0;
                slot_phase ^= 1;
            }
        }
        return;
    }

    if (warp == kConsumers + 1) {
        // ============================ loader ============================
        int slot = 0, buf = 0;
        uint32_t slot_phase = 0, buf_phase = 1;
        long long issued = 0;
        bool ok = true;
        for (;;) {
            ok = __all_sync(0xffffffffu, wait_phase(&p_meta[slot], slot_phase, a.batch.status, sSlow));
            Piece<ROWS>& p = pieces[slot];
            if (!ok || p.n_stages < 0) break;
            const int st0 = p.first_stage, st1 = st0 + p.n_stages, h = p.kv_head;
            const int* table = a.prefix_phase ? a.prefix_table : a.batch.table + (size_t)p.seq * a.batch.table_stride;
            const int n_table = a.prefix_phase ? (a.prefix_len + kPageTokens - 1) / kPageTokens : a.batch.table_stride;
            int pages = p.pages[lane], pages_at = st0 >> 1;  // 32 page numbers, one a lane
            for (int st = st0; st < st1; ++st) {
                const int j = st >> 1;
                if (j >= pages_at + 32) {
                    pages_at = j;
                    pages = j + lane < n_table ? table[j + lane] : -1;
                }
                int page = __shfl_sync(0xffffffffu, pages, j - pages_at);
                ok = __all_sync(0xffffffffu, wait_phase(&empty[buf], buf_phase, a.batch.status, sSlow));
                if (!ok) break;
                if (lane == 0) {
                    if ((unsigned)page >= (unsigned)a.pool.n_pages) page = 0;  // some page: rows that see it come out as NaN
                    uint8_t* dst = smem + buf * G::kBytes;
                    uint64_t* bar = &full[buf];
                    mbar_expect_tx(bar, G::kBytes);
                    const int hp = page * a.pool.n_kv + h, t0 = (st & 1) * kStageKeys;
                    const uint8_t* ph = a.pool.pages + (size_t)hp * PG::kHeadBytes;
                    if constexpr (KT == kKF16) {
                        tma4(dst, &maps.k, 0, 0, t0, hp, bar);
                        tma4(dst + kStageKeys * 128, &maps.k, 0, 1, t0, hp, bar);
                    } else {
                        tma3(dst, &maps.k, 0, t0, hp, bar);
                        bulk_load(dst + G::kOffKd, ph + PG::kOffKd + t0 * PG::kKdRow, kStageKeys * PG::kKdRow, bar);
                    }
                    if constexpr (VT == kVF16) {
                        tma4(dst + G::kOffV, &maps.v, 0, 0, PG::kOffVq / 256 + t0, hp, bar);
                        tma4(dst + G::kOffV + kStageKeys * 128, &maps.v, 0, 1, PG::kOffVq / 256 + t0, hp, bar);
                    } else {
                        tma3(dst + G::kOffV, &maps.v, 0, PG::kOffVq / PG::kVqRow + t0, hp, bar);
                        bulk_load(dst + G::kOffVd, ph + PG::kOffVd + t0 * PG::kVdRow, kStageKeys * PG::kVdRow, bar);
                    }
                    if constexpr (PG::kVhRow > 0)
                        bulk_load(dst + G::kOffVh, ph + PG::kOffVh + t0 * PG::kVhRow, kStageKeys * PG::kVhRow, bar);
                    if constexpr (PG::kVmRow > 0)
                        bulk_load(dst + G::kOffVm, ph + PG::kOffVm + t0 * PG::kVmRow, kStageKeys * PG::kVmRow, bar);
                }
                __syncwarp();
                ++issued;
                if (++buf == kStages) {
                    buf = 0;
                    buf_phase ^= 1;
                }
            }
            if (!ok) break;
            if (lane == 0) arrive(&p_empty[slot]);
            if (++slot == kSlots) {
                slot = 0;
                slot_phase ^= 1;
            }
        }
        // a wait gave up: the copies in flight land before the memory is given back
        for (long long k = max(0ll, issued - kStages); !ok && k < issued; ++k)
            mbar_wait_bounded(&full[k % kStages], (k / kStages) & 1, a.batch.status);
        return;
    }

    // ============================ consumers ============================
    const int g = lane >> 2, q = lane & 3;
    const bool formed = a.softcap > 0.0f || a.slopes;  // scores need more than a scale
    int buf = 0;                                       // the next stage's buffer and its phase
    uint32_t buf_phase = 0;
    // The barrier of the four consumer warps says whether a bounded wait of any of
    // them gave up; all leave then.  A warp whose wait failed still comes to the
    // next barrier, and so does one that has reached the end, so nobody is left.
    bool ok = true;
    auto consumers_sync = [&]() -> bool {
        int lost;
        asm volatile(
            "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 q, %1, 0;\n\tbarrier.cta.red.or.pred p, 1, 128, q;\n\tselp.b32 %0, 1, 0, p;\n\t}"
            : "=r"(lost)
            : "r"(ok ? 0 : 1)
            : "memory");
        return lost == 0;
    };
    int slot = 0;
    uint32_t slot_phase = 0;
    for (;;) {
        Piece<ROWS>& p = pieces[slot];
        ok = wait_phase(&p_full[slot], slot_phase, a.batch.status, sSlow);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok || p.n_stages < 0) {
            consumers_sync();
            return;
        }
        float o[8][NT][4];
        float ref[NT][2], l[NT][2], sc[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int t = 0; t < 8; ++t)
#pragma unroll
                for (int j = 0; j < 4; ++j) o[t][nt][j] = 0.0f;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                ref[nt][j] = -CUDART_INF_F;
                l[nt][j] = 0.0f;
                sc[nt][j] = p.scale[8 * nt + 2 * q + j];
            }
        }
        const uint8_t* sq = p.q + g * kQRow + 8 * q;  // this lane's operand: row g, dims 16 c + 4 q ..
        const int n_stages = p.n_stages;
        for (int i = 0; i < n_stages; ++i) {
            ok = wait_phase(&full[buf], buf_phase, a.batch.status, sSlow);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            const uint8_t* sb = smem + buf * G::kBytes;
            const int key0 = (p.first_stage + i) * kStageKeys;  // the stage's first key
            const int wk = warp * 32;                           // this warp's first key in it

            // ---- S^T = K Q^T: two tiles of 16 keys ----
            float s[2][NT][4];
#pragma unroll
            for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int j = 0; j < 4; ++j) s[mt][nt][j] = 0.0f;
            // ldmatrix rows of this lane: matrices 0, 1 = keys 0..7, 8..15 of a
            // chunk, 2, 3 = the next chunk
            const int lk = wk + (lane & 7) + ((lane >> 3) & 1) * 8, lc = lane >> 4;
            if constexpr (KT == kKF16) {
#pragma unroll
                for (int c = 0; c < 8; ++c) {  // 16 dims: two 8-dim chunks
                    uint2 qb[NT];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        // operand pairs (dims 16c + 2q, +1) and (16c + 8 + 2q, +1)
                        const uint8_t* r = p.q + (8 * nt + g) * kQRow + 32 * c + 4 * q;
                        qb[nt].x = *reinterpret_cast<const uint32_t*>(r);
                        qb[nt].y = *reinterpret_cast<const uint32_t*>(r + 16);
                    }
#pragma unroll
                    for (int mt = 0; mt < 2; ++mt) {
                        const int key = lk + 16 * mt, ch = (2 * c & 7) + lc;
                        uint32_t w[4];
                        ldsm4(smem_u32(sb + (c >> 2) * kStageKeys * 128 + key * 128 + ((ch ^ (key & 7)) << 4)), w);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) mma(s[mt][nt], w, qb[nt].x, qb[nt].y);
                    }
                }
            } else {
#pragma unroll
                for (int b = 0; b < kBlocks; ++b) {
                    uint2 qb[NT][2];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int c = 0; c < 2; ++c)
                            qb[nt][c] = *reinterpret_cast<const uint2*>(sq + 8 * nt * kQRow + 32 * (2 * b + c));
#pragma unroll
                    for (int mt = 0; mt < 2; ++mt) {
                        const int key = lk + 16 * mt, ch = 2 * b + lc;
                        uint32_t w[4], k0[4], k1[4];
                        ldsm4(smem_u32(sb + key * 128 + ((ch ^ (key & 7)) << 4)), w);
                        s8x4(w[0], 0x4140, 0x4342, k0[0], k0[2]);
                        s8x4(w[1], 0x4140, 0x4342, k0[1], k0[3]);
                        s8x4(w[2], 0x4140, 0x4342, k1[0], k1[2]);
                        s8x4(w[3], 0x4140, 0x4342, k1[1], k1[3]);
                        const __half* kd = reinterpret_cast<const __half*>(sb + G::kOffKd + (wk + 16 * mt + g) * 8) + b;
                        const float f0 = __half2float(kd[0]), f1 = __half2float(kd[8 * kBlocks]);  // keys g, g + 8
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            float c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                            mma(c, k0, qb[nt][0].x, qb[nt][0].y);
                            mma(c, k1, qb[nt][1].x, qb[nt][1].y);
                            s[mt][nt][0] = fmaf(f0, c[0], s[mt][nt][0]);
                            s[mt][nt][1] = fmaf(f0, c[1], s[mt][nt][1]);
                            s[mt][nt][2] = fmaf(f1, c[2], s[mt][nt][2]);
                            s[mt][nt][3] = fmaf(f1, c[3], s[mt][nt][3]);
                        }
                    }
                }
            }

            // ---- scores in the log2 domain; element j: key g + 8 (j / 2), row 2 q + (j & 1) ----
            const bool all_seen = key0 >= p.full_from && key0 + kStageKeys <= p.full_to;
            bool above = false;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                    for (int j = 0; j < 4; ++j) s[mt][nt][j] *= sc[nt][j & 1];
                if (formed) {
#pragma unroll
                    for (int jr = 0; jr < 2; ++jr) {
                        const int r = 8 * nt + 2 * q + jr;
                        const float slope = p.slope[r];
                        const int pos = p.pos[r];
#pragma unroll
                        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                            for (int jk = 0; jk < 2; ++jk)
                                s[mt][nt][2 * jk + jr] =
                                    score_log2(a, s[mt][nt][2 * jk + jr], slope, pos, key0 + wk + 16 * mt + 8 * jk + g);
                    }
                }
                if (!all_seen) {
#pragma unroll
                    for (int jr = 0; jr < 2; ++jr) {
                        const int first = p.first[8 * nt + 2 * q + jr], end = p.end[8 * nt + 2 * q + jr];
#pragma unroll
                        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                            for (int jk = 0; jk < 2; ++jk) {
                                const int key = key0 + wk + 16 * mt + 8 * jk + g;
                                if (key < first || key >= end) s[mt][nt][2 * jk + jr] = -CUDART_INF_F;
                            }
                    }
                }
#pragma unroll
                for (int jr = 0; jr < 2; ++jr) {
                    const float top = fmaxf(fmaxf(s[0][nt][jr], s[0][nt][2 + jr]), fmaxf(s[1][nt][jr], s[1][nt][2 + jr]));
                    above |= top > ref[nt][jr] + 9.0f;
                }
            }
            // The reference of a row is 6 below a maximum seen so far, and moves only
            // when a score passes it by 9: weights stay within 2^9, most near 2^6.
            if (__any_sync(0xffffffffu, above)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int jr = 0; jr < 2; ++jr) {
                        float top = fmaxf(fmaxf(s[0][nt][jr], s[0][nt][2 + jr]), fmaxf(s[1][nt][jr], s[1][nt][2 + jr]));
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16)) - 6.0f;
                        const float now = fmaxf(ref[nt][jr], top);
                        const float f = now == ref[nt][jr] ? 1.0f : exp2_fast(ref[nt][jr] - now);
                        ref[nt][jr] = now;
                        l[nt][jr] *= f;
#pragma unroll
                        for (int t = 0; t < 8; ++t) {
                            o[t][nt][jr] *= f;
                            o[t][nt][2 + jr] *= f;
                        }
                    }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int jr = 0; jr < 2; ++jr) {
                    const float r = ref[nt][jr] == -CUDART_INF_F ? 0.0f : ref[nt][jr];
#pragma unroll
                    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                        for (int jk = 0; jk < 2; ++jk) {
                            const float w = exp2_fast(s[mt][nt][2 * jk + jr] - r);
                            s[mt][nt][2 * jk + jr] = w;
                            l[nt][jr] += w;
                        }
                }

            // ---- O^T += V^T P^T, 16 keys at a time ----
            // weights with keys along the pair: [tile][nt][keys 2q,2q+1 | 8+2q, 8+2q+1],
            // and what their rounding to fp16 left
            uint32_t ph2[2][NT][2], pl2[2][NT][2];
#pragma unroll
            for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int jk = 0; jk < 2; ++jk) {
                        const float x = s[mt][nt][2 * jk], y = s[mt][nt][2 * jk + 1];
                        const __half2 hi = __floats2half2_rn(x, y);
                        ph2[mt][nt][jk] = movm(h2u(hi));
                        pl2[mt][nt][jk] = 0u;
                        if constexpr (PRECISE) {
                            const float2 f = __half22float2(hi);
                            pl2[mt][nt][jk] = movm(h2u(__floats2half2_rn(x - f.x, y - f.y)));
                        }
                    }
#pragma unroll
            for (int mt = 0; mt < 2; ++mt) {
                uint32_t ph[NT][2], pl[NT][2];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int jk = 0; jk < 2; ++jk) {
                        ph[nt][jk] = mt ? ph2[1][nt][jk] : ph2[0][nt][jk];
                        pl[nt][jk] = mt ? pl2[1][nt][jk] : pl2[0][nt][jk];
                    }
                // keys that do not exist hold anything: their scales (or values) become 0
                uint32_t keep[2] = {0xffffffffu, 0xffffffffu};
                if (!all_seen) {
#pragma unroll
                    for (int jk = 0; jk < 2; ++jk) {
                        const int key = key0 + wk + 16 * mt + 8 * jk + 2 * q;
                        keep[jk] = (key < p.n_keys ? 0xffffu : 0u) | (key + 1 < p.n_keys ? 0xffff0000u : 0u);
                    }
                }
                uint4 dv[2], mv[2];  // four block scales (minima) of keys 2q and 2q + 1 of each half
                if constexpr (VT != kVF16) {
#pragma unroll
                    for (int jk = 0; jk < 2; ++jk) {
                        dv[jk] = *reinterpret_cast<const uint4*>(sb + G::kOffVd + (wk + 16 * mt + 8 * jk + 2 * q) * 8);
                        if constexpr (v_has_min(VT))
                            mv[jk] = *reinterpret_cast<const uint4*>(sb + G::kOffVm + (wk + 16 * mt + 8 * jk + 2 * q) * 8);
                    }
                }
                // block b of a key pair: (key 2q, key 2q + 1)
                auto pair = [&](const uint4& v, int b) -> uint32_t {
                    return (b < 2) ? __byte_perm(v.x, v.z, (b & 1) ? 0x7632 : 0x5410)
                                   : __byte_perm(v.y, v.w, (b & 1) ? 0x7632 : 0x5410);
                };
#pragma unroll
                for (int b = 0; b < kBlocks; ++b) {
                    uint32_t bh[NT][2], bl[NT][2];
                    __half2 dvp[2], mvp[2];
                    if constexpr (VT != kVF16) {
#pragma unroll
                        for (int jk = 0; jk < 2; ++jk) {
                            dvp[jk] = u2h(pair(dv[jk], b) & keep[jk]);
                            if constexpr (v_has_min(VT)) mvp[jk] = u2h(pair(mv[jk], b) & keep[jk]);
                        }
                    }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int jk = 0; jk < 2; ++jk) {
                            if constexpr (v_a_is_p(VT)) {
                                bh[nt][jk] = ph[nt][jk];
                                bl[nt][jk] = pl[nt][jk];
                            } else {
                                const __half2 hi = __hmul2(u2h(ph[nt][jk]), dvp[jk]);
                                bh[nt][jk] = h2u(hi);
                                if constexpr (PRECISE)  // the product's own error (exact by fma) and the low term
                                    bl[nt][jk] = h2u(__hfma2(u2h(pl[nt][jk]), dvp[jk], __hfma2(u2h(ph[nt][jk]), dvp[jk], __hneg2(hi))));
                            }
                        }
                    // the block's two tiles of 16 dims: rows g, g + 8 of tile e
                    uint32_t va[2][4];
                    if constexpr (VT == kVF16) {
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int ch = 2 * (2 * b + e);  // 8-dim chunk; matrices: keys 0..7, 8..15 of it, then of the next
                            const int key = wk + 16 * mt + (lane & 7) + ((lane >> 3) & 1) * 8, cl = (ch & 7) + (lane >> 4);
                            uint32_t w[4];
                            ldsm4t(smem_u32(sb + G::kOffV + (ch >> 3) * kStageKeys * 128 + key * 128 + ((cl ^ (key & 7)) << 4)), w);
                            va[e][0] = w[0] & keep[0];
                            va[e][1] = w[2] & keep[0];
                            va[e][2] = w[1] & keep[1];
                            va[e][3] = w[3] & keep[1];
                        }
                    } else if constexpr (VT == kVQ8_0) {
                        const int key = wk + 16 * mt + (lane & 7) + ((lane >> 3) & 1) * 8, ch = 2 * b + (lane >> 4);
                        uint32_t w[4];
                        ldsm4t(smem_u32(sb + G::kOffV + key * 128 + ((ch ^ (key & 7)) << 4)), w);
#pragma unroll
                        for (int e = 0; e < 2; ++e) {  // word: (key 2q: dims 2g, 2g+1 | key 2q+1: the same)
                            s8x4(w[2 * e], 0x4240, 0x4341, va[e][0], va[e][1]);
                            s8x4(w[2 * e + 1], 0x4240, 0x4341, va[e][2], va[e][3]);
                        }
                    } else {
                        uint32_t w[2];
                        const int key = wk + 16 * mt + (lane & 7) + ((lane >> 3) & 1) * 8, ch = b;
                        asm volatile("ldmatrix.sync.aligned.m8n8.x2.trans.shared.b16 {%0, %1}, [%2];"
                                     : "=r"(w[0]), "=r"(w[1])
                                     : "r"(smem_u32(sb + G::kOffV + key * 64 + ((ch ^ ((key >> 1) & 3)) << 4))) : "memory");
#pragma unroll
                        for (int jk = 0; jk < 2; ++jk) {
                            // word: (key 2q: bytes 2g, 2g+1 | key 2q+1: the same); a byte's low nibble is
                            // dim 2g (+1), its high nibble dim 16 + 2g (+1)
                            uint32_t f[2][2] = {{0u, 0u}, {0u, 0u}};  // fifth bits in place, [nibble][byte]
                            if constexpr (v_has_fifth(VT)) {
                                const uint8_t* hp = sb + G::kOffVh + (wk + 16 * mt + 8 * jk + 2 * q) * 16 + 4 * b;
                                const uint32_t h0 = *reinterpret_cast<const uint32_t*>(hp) >> (2 * g);
                                const uint32_t h1 = *reinterpret_cast<const uint32_t*>(hp + 16) >> (2 * g);
                                const uint32_t u = __byte_perm(h0, h1, 0x5410), v = __byte_perm(h0, h1, 0x7632);
                                f[0][0] = (u << 4) & 0x00100010u;
                                f[0][1] = (u << 3) & 0x00100010u;
                                f[1][0] = (v << 8) & 0x01000100u;
                                f[1][1] = (v << 7) & 0x01000100u;
                            }
                            constexpr float kZero = v_has_min(VT) ? 0.0f : (VT == kVQ5_0 ? 16.0f : 8.0f);
                            const __half2 z0 = __float2half2_rn(1024.0f + kZero), z1 = __float2half2_rn(-64.0f - kZero);
                            const __half2 six = __float2half2_rn(0.0625f);
                            const uint32_t y = w[jk] >> 8;
                            __half2 c[2][2];
                            c[0][0] = __hsub2(u2h((w[jk] & 0x000f000fu) | 0x64006400u | f[0][0]), z0);
                            c[0][1] = __hsub2(u2h((y & 0x000f000fu) | 0x64006400u | f[0][1]), z0);
                            c[1][0] = __hfma2(u2h((w[jk] & 0x00f000f0u) | 0x64006400u | f[1][0]), six, z1);
                            c[1][1] = __hfma2(u2h((y & 0x00f000f0u) | 0x64006400u | f[1][1]), six, z1);
#pragma unroll
                            for (int e = 0; e < 2; ++e)
#pragma unroll
                                for (int u = 0; u < 2; ++u) {
                                    if constexpr (v_has_min(VT)) c[e][u] = __hfma2(c[e][u], dvp[jk], mvp[jk]);
                                    va[e][2 * jk + u] = h2u(c[e][u]);
                                }
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 2; ++e)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            mma(o[2 * b + e][nt], va[e], bh[nt][0], bh[nt][1]);
                            if constexpr (PRECISE) mma(o[2 * b + e][nt], va[e], bl[nt][0], bl[nt][1]);
                        }
                }
            }
            __syncwarp();
            if (lane == 0) arrive(&empty[buf]);
            if (++buf == kStages) {
                buf = 0;
                buf_phase ^= 1;
            }
        }

        // ---- the piece's end ----
        // What the prefix left for this warp's two rows of 8 nt .. + 7, on its way early
        float4 pacc[2];
        float2 pml[2];
        auto fetch_prior = [&](int nt) {
#pragma unroll
            for (int rr = 0; rr < 2; ++rr) {
                const int pr = 8 * nt + warp + kConsumers * rr;
                pml[rr] = make_float2(-CUDART_INF_F, 0.0f);
                pacc[rr] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (!a.prefix_phase && a.prefix_len > 0 && pr < p.rows && p.token[pr] >= 0) {
                    const size_t at = (size_t)p.token[pr] * a.n_qh + p.head[pr];
                    pml[rr] = a.prior_ml[at];
                    pacc[rr] = reinterpret_cast<const float4*>(a.prior_acc)[at * 32 + lane];
                }
            }
        };
        // joins the four warps' sums of those rows from the join buffer, lane = dims
        // 4 lane .. + 3, and ends them or keeps the CTA's record
        auto join_warps = [&](int nt, bool record) {
#pragma unroll
            for (int rr = 0; rr < 2; ++rr) {
                const int r = warp + kConsumers * rr, pr = 8 * nt + r;
                if (pr >= p.rows || p.token[pr] < 0) continue;
                float M = -CUDART_INF_F, L = 0.0f;
                float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                for (int w = 0; w < kConsumers; ++w)
                    join(acc, M, L, *reinterpret_cast<const float4*>(red + (w * 8 + r) * kRedRow + 4 * lane), sml[(w * 8 + r) * 2],
                         sml[(w * 8 + r) * 2 + 1]);
                if (!record) {
                    join(acc, M, L, pacc[rr], pml[rr].x, pml[rr].y);
                    end_row<VT, KT>(a, p.seq, p.token[pr], p.head[pr], acc, M, L, sSlow);
                } else {
                    float* rec = a.records + ((size_t)(blockIdx.x * 2 + p.slot) * kFewRowsMax + pr) * kRecordFloats;
                    *reinterpret_cast<float4*>(rec + 4 * lane) = acc;
                    if (lane == 0) *reinterpret_cast<float2*>(rec + 128) = make_float2(M, L);
                }
            }
        };
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            if (8 * nt >= p.rows) break;  // uniform
            if (p.slot < 0) fetch_prior(nt);
#pragma unroll
            for (int jr = 0; jr < 2; ++jr) {
                float sum = l[nt][jr];
                sum += __shfl_xor_sync(0xffffffffu, sum, 4);
                sum += __shfl_xor_sync(0xffffffffu, sum, 8);
                sum += __shfl_xor_sync(0xffffffffu, sum, 16);
                if (g == 0) {
                    sml[(warp * 8 + 2 * q + jr) * 2] = ref[nt][jr];
                    sml[(warp * 8 + 2 * q + jr) * 2 + 1] = (p.nan_rows >> (8 * nt + 2 * q + jr)) & 1u ? CUDART_NAN_F : sum;
                }
                float* dst = red + (warp * 8 + 2 * q + jr) * kRedRow;
#pragma unroll
                for (int t = 0; t < 8; ++t) {
                    if constexpr (VT == kVF16) {  // tile t: dims 16 t + g and 16 t + 8 + g
                        dst[16 * t + g] = o[t][nt][jr];
                        dst[16 * t + 8 + g] = o[t][nt][2 + jr];
                    } else {  // dims 16 t + 2 g, + 1
                        *reinterpret_cast<float2*>(dst + 16 * t + 2 * g) = make_float2(o[t][nt][jr], o[t][nt][2 + jr]);
                    }
                }
            }
            if (!consumers_sync()) return;
            join_warps(nt, p.slot >= 0);
            if (!consumers_sync()) return;
        }
        if (p.slot >= 0) {
            // ---- a shared unit: the last CTA to arrive joins the records.  Each warp
            // takes every fourth record, four rows of four records in flight
            // (the barrier orders the warps' records before the thread's release) ----
            if (!consumers_sync()) return;
            if (tid == 0) {
                int before;
                asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], 1;" : "=r"(before) : "l"(a.counters + p.cta0) : "memory");
                const bool last = before == p.n_ctas - 1;
                if (last) a.counters[p.cta0] = 0;  // ready for the next call
                *sLast = last;
            }
            if (!consumers_sync()) return;
            if (*sLast) {
                const int n = p.n_ctas, cta0 = p.cta0, rows = p.rows;
                constexpr int kRec = 4, kRow = 4;
#pragma unroll 1
                for (int nt = 0; 8 * nt < rows; ++nt) {
                    fetch_prior(nt);
#pragma unroll 1
                    for (int r0 = 0; r0 < 8 && 8 * nt + r0 < rows; r0 += kRow) {
                        float4 acc[kRow];
                        float M[kRow], L[kRow];
#pragma unroll
                        for (int k = 0; k < kRow; ++k) {
                            acc[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                            M[k] = -CUDART_INF_F;
                            L[k] = 0.0f;
                        }
#pragma unroll 1
                        for (int c0 = warp; c0 < n; c0 += kConsumers * kRec) {
                            float4 v[kRec][kRow];
                            float2 ml[kRec][kRow];
#pragma unroll
                            for (int b = 0; b < kRec; ++b) {
                                const int c = c0 + kConsumers * b;
                                // the first CTA began the unit, the others continue it
                                const float* rec = a.records +
                                    ((size_t)((cta0 + min(c, n - 1)) * 2 + (c == 0 ? 1 : 0)) * kFewRowsMax + 8 * nt + r0) * kRecordFloats;
#pragma unroll
                                for (int k = 0; k < kRow; ++k) {
                                    v[b][k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                                    ml[b][k] = make_float2(-CUDART_INF_F, 0.0f);
                                    if (c < n && 8 * nt + r0 + k < rows) {
                                        v[b][k] = __ldcg(reinterpret_cast<const float4*>(rec + k * kRecordFloats) + lane);
                                        ml[b][k] = __ldcg(reinterpret_cast<const float2*>(rec + k * kRecordFloats + 128));
                                    }
                                }
                            }
#pragma unroll
                            for (int b = 0; b < kRec; ++b)
#pragma unroll
                                for (int k = 0; k < kRow; ++k) join(acc[k], M[k], L[k], v[b][k], ml[b][k].x, ml[b][k].y);
                        }
#pragma unroll
                        for (int k = 0; k < kRow; ++k) {
                            *reinterpret_cast<float4*>(red + (warp * 8 + r0 + k) * kRedRow + 4 * lane) = acc[k];
                            if (lane == 0) {
                                sml[(warp * 8 + r0 + k) * 2] = M[k];
                                sml[(warp * 8 + r0 + k) * 2 + 1] = L[k];
                            }
                        }
                    }
                    if (!consumers_sync()) return;
                    join_warps(nt, false);
                    if (!consumers_sync()) return;
                }
            }
        }
        if (!consumers_sync()) return;  // sLast and the join buffer are free again
        if (lane == 0) arrive(&p_empty[slot]);
        if (++slot == kSlots) {
            slot = 0;
            slot_phase ^= 1;
        }
    }
}

template <int VT, int KT, int NT, bool PRECISE>
cudaError_t launch(const AttendPagesArgs& a, const PageMaps& maps, int n_sms, cudaStream_t s) {
    using G = Geo<VT, KT, NT>;
    // the shared-memory opt-in is per device
    static std::atomic<unsigned long long> configured{0};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev >= 64 || !(configured.load(std::memory_order_acquire) & (1ull << dev))) {
        const cudaError_t e = cudaFuncSetAttribute(attend_few_kernel<VT, KT, NT, PRECISE>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)G::kSmem);
        if (e != cudaSuccess) return e;
        if (dev < 64) configured.fetch_or(1ull << dev, std::memory_order_acq_rel);
    }
    attend_few_kernel<VT, KT, NT, PRECISE><<<std::min(kFewCtas, n_sms * G::kPerSm), kThreads, G::kSmem, s>>>(a, maps);
    return cudaGetLastError();
}

template <int VT, int KT>
cudaError_t by_rows(const AttendPagesArgs& a, const PageMaps& maps, int unit_rows, int n_sms, cudaStream_t s) {
    if (unit_rows <= 8)
        return a.precise ? launch<VT, KT, 1, true>(a, maps, n_sms, s) : launch<VT, KT, 1, false>(a, maps, n_sms, s);
    return a.precise ? launch<VT, KT, 2, true>(a, maps, n_sms, s) : launch<VT, KT, 2, false>(a, maps, n_sms, s);
}

}  // namespace

cudaError_t launch_attend_few(const AttendPagesArgs& a, const PageMaps& maps, int unit_rows, int n_sms, cudaStream_t s) {
    if (a.pool.k_type == kKF16) return by_rows<kVF16, kKF16>(a, maps, unit_rows, n_sms, s);
    switch (a.pool.v_type) {
        case kVF16: return by_rows<kVF16, kKQ8_0>(a, maps, unit_rows, n_sms, s);
        case kVQ4_1: return by_rows<kVQ4_1, kKQ8_0>(a, maps, unit_rows, n_sms, s);
        case kVQ5_0: return by_rows<kVQ5_0, kKQ8_0>(a, maps, unit_rows, n_sms, s);
        case kVQ5_1: return by_rows<kVQ5_1, kKQ8_0>(a, maps, unit_rows, n_sms, s);
        case kVQ8_0: return by_rows<kVQ8_0, kKQ8_0>(a, maps, unit_rows, n_sms, s);
        default: return by_rows<kVQ4_0, kKQ8_0>(a, maps, unit_rows, n_sms, s);
    }
}

}  // namespace kvs
