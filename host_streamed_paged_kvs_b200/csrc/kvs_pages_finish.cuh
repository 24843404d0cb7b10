// kvs_pages_finish.cuh -- how a row of the page attention ends: the join of its
// records, the division by the sum of weights, and the recomputation of rows
// whose sums an unseen key's value spoiled.  Internal to libkvs.
#pragma once

#include <cuda_bf16.h>
#include <math_constants.h>

#include "kvs_pages.h"
#include "kvs_pages_wait.h"
#include "kvs_ptx.cuh"

namespace kvs {

// Waits for an mbarrier phase, for at most about 10 s beside the time that other
// warps of the block take to recompute rows (*busy counts them).  The clock is
// read only after many failed tries: reading it costs more than the wait for a
// barrier that is nearly always complete.
__device__ __forceinline__ bool wait_phase(uint64_t* bar, uint32_t parity, int* err, const volatile int* busy) {
    WaitClock clock;
    for (uint32_t it = 0;; ++it) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((it & 1023) == 1023 && clock.expired(globaltimer_ns(), *busy != 0)) {
            if (err) atomicOr(err, kErrWaitTimeout);
            return false;
        }
    }
}

// Whether a row that sees the keys first .. end - 1 (of this phase's table) sees
// one beyond the table, or one of the keys from .. to - 1 whose page is not in the
// pool.  Called where some page number is known to be bad, so plain loads will do.
__device__ __forceinline__ bool sees_bad_page(const int* table, int n_table, int n_pages, int first, int end, int from, int to) {
    if (max((long long)first, (long long)n_table * kPageTokens) < end) return true;
    const int k0 = max(first, from), k1 = min(end, to);
    if (k0 < k1)
        for (int j = k0 / kPageTokens; j <= (k1 - 1) / kPageTokens; ++j)
            if (j >= n_table || (unsigned)table[j] >= (unsigned)n_pages) return true;
    return false;
}

// Value d of the K or V row of token t in a page head, fp32 (exact).
template <int VT, int KT>
__device__ __forceinline__ float k_value(const uint8_t* ph, int t, int d) {
    using G = PageGeom<VT, KT>;
    if constexpr (KT == kKF16) return __half2float(reinterpret_cast<const __half*>(ph)[t * 128 + d]);
    else return __half2float(*reinterpret_cast<const __half*>(ph + G::kOffKd + t * 8 + 2 * (d >> 5))) *
                static_cast<float>(static_cast<int8_t>(ph[t * 128 + d]));
}
template <int VT, int KT>
__device__ __forceinline__ float v_value(const uint8_t* ph, int t, int d) {
    using G = PageGeom<VT, KT>;
    if constexpr (VT == kVF16) return __half2float(reinterpret_cast<const __half*>(ph + G::kOffVq)[t * 128 + d]);
    else {
        const float s = __half2float(*reinterpret_cast<const __half*>(ph + G::kOffVd + t * 8 + 2 * (d >> 5)));
        if constexpr (VT == kVQ8_0) return s * static_cast<float>(static_cast<int8_t>(ph[G::kOffVq + t * 128 + d]));
        else {
            const int b = d >> 5, j = d & 31;
            int q = (ph[G::kOffVq + t * 64 + b * 16 + (j & 15)] >> (j < 16 ? 0 : 4)) & 15;
            if constexpr (v_has_fifth(VT))
                q |= ((*reinterpret_cast<const uint32_t*>(ph + G::kOffVh + t * 16 + 4 * b) >> j) & 1u) << 4;
            if constexpr (v_has_min(VT))
                return fmaf(s, static_cast<float>(q), __half2float(*reinterpret_cast<const __half*>(ph + G::kOffVm + t * 8 + 2 * b)));
            else return s * static_cast<float>(q - (VT == kVQ5_0 ? 16 : 8));
        }
    }
}

template <int DT>
__device__ __forceinline__ float one_value(const void* p, long long at) {
    if constexpr (DT == kDtF16) return __half2float(static_cast<const __half*>(p)[at]);
    else return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[at]);
}

// One row of the result by one warp, straight from its definition and only
// over the keys that it sees.  The tensor-core products multiply every value
// of a tile, with weight 0 where a row does not see the key, and 0 times an
// infinity or NaN is NaN; products of weights and scales may also pass fp16's
// range.  Rows that end non-finite with a finite sum of weights come here, so
// that what they do not see does not count.  Slow (a few us per 32 keys), and
// no call with finite, moderate values reaches it.  busy: counts the block's warps
// that are here, for those that wait; null where none does.
template <int VT, int KT>
__device__ __noinline__ float4 slow_row(const AttendPagesArgs& a, int seq, int row, int head, int* busy) {
    using G = PageGeom<VT, KT>;
    const int lane = threadIdx.x & 31, h = head / a.group;
    if (busy && lane == 0) atomicAdd(busy, 1);
    const RowView v = row_view(a, seq, row);
    const float slope = a.slopes ? a.slopes[head] : 0.0f;
    auto head_of = [&](int key) -> const uint8_t* {
        const int own = key - a.prefix_len;
        int page = -1;
        if (own < 0) page = a.prefix_table[key >> 8];
        else if ((own >> 8) < a.batch.table_stride) page = a.batch.table[(size_t)seq * a.batch.table_stride + (own >> 8)];
        if ((unsigned)page >= (unsigned)a.pool.n_pages) return nullptr;
        return a.pool.pages + ((size_t)page * a.pool.n_kv + h) * G::kHeadBytes;
    };
    auto token_of = [&](int key) { return (key < a.prefix_len ? key : key - a.prefix_len) & 255; };
    auto score = [&](int key) {
        const uint8_t* ph = head_of(key);
        if (!ph) return CUDART_NAN_F;
        const int t = token_of(key);
        const long long at = row * a.q.row + head * a.q.head;
        float s = 0.0f;
        for (int d = 0; d < kHeadDim; ++d) {
            const float q = a.q_dtype == kDtF16 ? one_value<kDtF16>(a.q.p, at + d) : one_value<kDtBF16>(a.q.p, at + d);
            s = fmaf(q, k_value<VT, KT>(ph, t, d), s);
        }
        return score_log2(a, s * a.scale, slope, v.pos, key);
    };
    float m = -CUDART_INF_F;
    for (int key = v.first + lane; key < v.end; key += 32) m = fmaxf(m, score(key));
#pragma unroll
    for (int off = 16; off; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    float l = 0.0f;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int k0 = v.first; k0 < v.end; k0 += 32) {
        const float p = k0 + lane < v.end ? exp2_fast(score(k0 + lane) - m) : 0.0f;
        l += p;
        for (int j = 0; j < 32 && k0 + j < v.end; ++j) {
            const float pj = __shfl_sync(0xffffffffu, p, j);
            const uint8_t* ph = head_of(k0 + j);
            if (!ph) continue;  // its score was NaN already
            const int t = token_of(k0 + j);
            o.x = fmaf(pj, v_value<VT, KT>(ph, t, 4 * lane), o.x);
            o.y = fmaf(pj, v_value<VT, KT>(ph, t, 4 * lane + 1), o.y);
            o.z = fmaf(pj, v_value<VT, KT>(ph, t, 4 * lane + 2), o.z);
            o.w = fmaf(pj, v_value<VT, KT>(ph, t, 4 * lane + 3), o.w);
        }
    }
#pragma unroll
    for (int off = 16; off; off >>= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
    const float r = 1.0f / l;
    if (busy && lane == 0) atomicAdd(busy, -1);
    return make_float4(o.x * r, o.y * r, o.z * r, o.w * r);
}

// four values of the result
__device__ __forceinline__ void store_out4_at(const AttendPagesArgs& a, long long to, const float4& o) {
    if (a.out_dtype == kDtF32) {
        *reinterpret_cast<float4*>(static_cast<float*>(a.out.p) + to) = o;
        return;
    }
    uint2 w;
    if (a.out_dtype == kDtF16) {
        *reinterpret_cast<__half2*>(&w.x) = __floats2half2_rn(o.x, o.y);
        *reinterpret_cast<__half2*>(&w.y) = __floats2half2_rn(o.z, o.w);
    } else {
        *reinterpret_cast<__nv_bfloat162*>(&w.x) = __floats2bfloat162_rn(o.x, o.y);
        *reinterpret_cast<__nv_bfloat162*>(&w.y) = __floats2bfloat162_rn(o.z, o.w);
    }
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out.p) + to) = w;
}

__device__ __forceinline__ void store_out4(const AttendPagesArgs& a, int row, int head, int d, const float4& o) {
    store_out4_at(a, row * a.out.row + head * a.out.head + d, o);
}

// (acc, M, L) += (b, m, l): records relative to 2^M and 2^m
__device__ __forceinline__ void join(float4& acc, float& M, float& L, const float4& b, float m, float l) {
    const float top = fmaxf(M, m);
    const float wa = M == top ? 1.0f : exp2_fast(M - top), wb = m == top ? 1.0f : exp2_fast(m - top);
    acc.x = acc.x * wa + b.x * wb;
    acc.y = acc.y * wa + b.y * wb;
    acc.z = acc.z * wa + b.z * wb;
    acc.w = acc.w * wa + b.w * wb;
    L = L * wa + l * wb;
    M = top;
}

// The end of one row, by a whole warp: lane holds sums of dims 4 lane .. + 3
// relative to 2^M, L the sum of weights (0: the row sees nothing), the prefix's
// part joined.  The prefix phase keeps the record, the own phase divides and
// writes.  busy as for slow_row.
template <int VT, int KT>
__device__ __forceinline__ void end_row(const AttendPagesArgs& a, int seq, int row, int head, const float4& acc, float M, float L, int* busy) {
    const int lane = threadIdx.x & 31;
    const size_t at = (size_t)row * a.n_qh + head;
    if (a.prefix_phase) {
        reinterpret_cast<float4*>(a.prior_acc)[at * 32 + lane] = acc;
        if (lane == 0) a.prior_ml[at] = make_float2(M, L);
        return;
    }
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (L != 0.0f) {
        const float r = 1.0f / L;
        o = make_float4(acc.x * r, acc.y * r, acc.z * r, acc.w * r);
        // inf - inf and 0 * inf make NaN, so a sum that is finite times 0 is 0
        const bool bad = !((acc.x + acc.y + acc.z + acc.w) * 0.0f == 0.0f);
        if (__any_sync(0xffffffffu, bad) && L * 0.0f == 0.0f) o = slow_row<VT, KT>(a, seq, row, head, busy);
    }
    store_out4(a, row, head, 4 * lane, o);
    if (a.lse && lane == 0) a.lse[at] = L == 0.0f ? -CUDART_INF_F : (M + log2f(L)) * 0.69314718055994531f;
}

// The same, with the prefix's part fetched here.
template <int VT, int KT>
__device__ __forceinline__ void finish_row(const AttendPagesArgs& a, int seq, int row, int head, float4 acc, float M, float L) {
    if (!a.prefix_phase && a.prefix_len > 0) {
        const size_t at = (size_t)row * a.n_qh + head;
        const float2 ml = a.prior_ml[at];
        join(acc, M, L, reinterpret_cast<const float4*>(a.prior_acc)[at * 32 + (threadIdx.x & 31)], ml.x, ml.y);
    }
    end_row<VT, KT>(a, seq, row, head, acc, M, L, nullptr);
}

}  // namespace kvs
