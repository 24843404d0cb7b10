// kvs_pages.cu -- append with rotation and read-back for a batch of sequences
// over caller-owned pages (kvs_append_pages, kvs_read_pages).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kvs_pages.h"

namespace kvs {
namespace {

// ---- four consecutive values of a row <-> four floats ----
template <int DT>
__device__ __forceinline__ void load4(const void* base, long long at, float (&x)[4]) {
    if constexpr (DT == kDtF32) {
        const float4 v = *reinterpret_cast<const float4*>(static_cast<const float*>(base) + at);
        x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
    } else {
        const uint2 v = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(base) + at);
        float2 a, b;
        if constexpr (DT == kDtF16) {
            a = __half22float2(*reinterpret_cast<const __half2*>(&v.x));
            b = __half22float2(*reinterpret_cast<const __half2*>(&v.y));
        } else {
            a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&v.x));
            b = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&v.y));
        }
        x[0] = a.x; x[1] = a.y; x[2] = b.x; x[3] = b.y;
    }
}
template <int DT>
__device__ __forceinline__ void store4(void* base, long long at, const float (&x)[4]) {
    if constexpr (DT == kDtF32) {
        *reinterpret_cast<float4*>(static_cast<float*>(base) + at) = make_float4(x[0], x[1], x[2], x[3]);
    } else {
        uint2 v;
        if constexpr (DT == kDtF16) {
            *reinterpret_cast<__half2*>(&v.x) = __floats2half2_rn(x[0], x[1]);
            *reinterpret_cast<__half2*>(&v.y) = __floats2half2_rn(x[2], x[3]);
        } else {
            *reinterpret_cast<__nv_bfloat162*>(&v.x) = __floats2bfloat162_rn(x[0], x[1]);
            *reinterpret_cast<__nv_bfloat162*>(&v.y) = __floats2bfloat162_rn(x[2], x[3]);
        }
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(base) + at) = v;
    }
}

// the same from 64 bits, each value rounded once (a value rounded to binary32 on
// the way may fall on the middle of two numbers of the type)
template <int DT>
__device__ __forceinline__ void store4(void* base, long long at, const double (&x)[4]) {
    if constexpr (DT == kDtF32) {
        *reinterpret_cast<float4*>(static_cast<float*>(base) + at) = make_float4((float)x[0], (float)x[1], (float)x[2], (float)x[3]);
    } else {
        uint2 v;
        if constexpr (DT == kDtF16) {
            *reinterpret_cast<__half2*>(&v.x) = __halves2half2(__double2half(x[0]), __double2half(x[1]));
            *reinterpret_cast<__half2*>(&v.y) = __halves2half2(__double2half(x[2]), __double2half(x[3]));
        } else {
            *reinterpret_cast<__nv_bfloat162*>(&v.x) = __halves2bfloat162(__double2bfloat16(x[0]), __double2bfloat16(x[1]));
            *reinterpret_cast<__nv_bfloat162*>(&v.y) = __halves2bfloat162(__double2bfloat16(x[2]), __double2bfloat16(x[3]));
        }
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(base) + at) = v;
    }
}

__device__ __forceinline__ uint2 pack_half4(const float (&x)[4]) {
    uint2 v;
    *reinterpret_cast<__half2*>(&v.x) = __floats2half2_rn(x[0], x[1]);
    *reinterpret_cast<__half2*>(&v.y) = __floats2half2_rn(x[2], x[3]);
    return v;
}

// ---- block quantizers: lane l of the warp has values 4l..4l+3 of the row, 8
// lanes a 32-value block.  The same rules as the handle's append: decisions in
// binary32 with correctly rounded division, scales stored as fp16. ----
__device__ __forceinline__ uint32_t quant_q8(const float (&x)[4], float& d) {
    float amax = fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3])));
#pragma unroll
    for (int off = 1; off <= 4; off <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
    d = __fdiv_rn(amax, 127.0f);
    uint32_t w = 0;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const int q = d != 0.0f ? static_cast<int>(roundf(__fdiv_rn(x[u], d))) : 0;
        w |= (static_cast<uint32_t>(q) & 0xffu) << (8 * u);
    }
    return w;
}

// codes of the 4- and 5-bit types: low nibbles one per byte, fifth bits at 4i + u of the block's word
template <int VT>
__device__ __forceinline__ void quant_low(const float (&x)[4], int i, uint32_t& codes, uint32_t& high, float& d, float& lo) {
    codes = high = 0;
    lo = 0.0f;
    int q[4];
    if constexpr (v_has_min(VT)) {
        constexpr int kL = PageGeom<VT>::kLevels;
        // first index on ties only tells +0 from -0
        float mn = x[0], mx = x[0];
        int imn = 4 * i;
#pragma unroll
        for (int u = 1; u < 4; ++u) {
            if (x[u] < mn) { mn = x[u]; imn = 4 * i + u; }
            if (x[u] > mx) mx = x[u];
        }
#pragma unroll
        for (int off = 1; off <= 4; off <<= 1) {
            const float pm = __shfl_xor_sync(0xffffffffu, mn, off);
            const int pi = __shfl_xor_sync(0xffffffffu, imn, off);
            const float px = __shfl_xor_sync(0xffffffffu, mx, off);
            if (pm < mn || (pm == mn && pi < imn)) { mn = pm; imn = pi; }
            if (px > mx) mx = px;
        }
        lo = mn;
        d = __fdiv_rn(__fsub_rn(mx, mn), static_cast<float>(kL));
#pragma unroll
        for (int u = 0; u < 4; ++u)
            q[u] = d != 0.0f ? min(kL, static_cast<int>(__fadd_rn(__fdiv_rn(__fsub_rn(x[u], mn), d), 0.5f))) : 0;
    } else {
        constexpr int kHalf = VT == kVQ5_0 ? 16 : 8;
        // the value of largest magnitude, first index on ties
        float va = 0.0f, vm = 0.0f;
        int vi = 1 << 30;
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (fabsf(x[u]) > va) { va = fabsf(x[u]); vm = x[u]; vi = 4 * i + u; }
#pragma unroll
        for (int off = 1; off <= 4; off <<= 1) {
            const float pa = __shfl_xor_sync(0xffffffffu, va, off);
            const float pm = __shfl_xor_sync(0xffffffffu, vm, off);
            const int pi = __shfl_xor_sync(0xffffffffu, vi, off);
            if (pa > va || (pa == va && pi < vi)) { va = pa; vm = pm; vi = pi; }
        }
        d = __fdiv_rn(vm, static_cast<float>(-kHalf));
#pragma unroll
        for (int u = 0; u < 4; ++u)
            q[u] = d != 0.0f ? min(2 * kHalf - 1, static_cast<int>(__fadd_rn(__fdiv_rn(x[u], d), kHalf + 0.5f))) : kHalf;
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        codes |= static_cast<uint32_t>(q[u] & 15) << (8 * u);
        high |= static_cast<uint32_t>((q[u] >> 4) & 1) << (4 * i + u);
    }
}

// One K row and one V row (lane: values 4 lane ..) into token t of a page head.
// `write` is uniform over the warp; the shuffles run either way.
template <int VT, int KT>
__device__ __forceinline__ void store_kv(uint8_t* ph, int t, const float (&xk)[4], const float (&xv)[4], bool write) {
    using G = PageGeom<VT, KT>;
    const int lane = threadIdx.x & 31, b = lane >> 3, i = lane & 7;
    if constexpr (KT == kKF16) {
        if (write) *reinterpret_cast<uint2*>(ph + t * G::kKqRow + 8 * lane) = pack_half4(xk);
    } else {
        float d;
        const uint32_t w = quant_q8(xk, d);
        if (write) {
            *reinterpret_cast<uint32_t*>(ph + t * G::kKqRow + 4 * lane) = w;
            if (i == 0) *reinterpret_cast<__half*>(ph + G::kOffKd + t * 8 + 2 * b) = __float2half_rn(d);
        }
    }
    if constexpr (VT == kVF16) {
        if (write) *reinterpret_cast<uint2*>(ph + G::kOffVq + t * G::kVqRow + 8 * lane) = pack_half4(xv);
    } else if constexpr (VT == kVQ8_0) {
        float d;
        const uint32_t w = quant_q8(xv, d);
        if (write) {
            *reinterpret_cast<uint32_t*>(ph + G::kOffVq + t * G::kVqRow + 4 * lane) = w;
            if (i == 0) *reinterpret_cast<__half*>(ph + G::kOffVd + t * 8 + 2 * b) = __float2half_rn(d);
        }
    } else {
        uint32_t codes, high;
        float d, lo;
        quant_low<VT>(xv, i, codes, high, d, lo);
        // byte j of a block: code j low, code j + 16 (four lanes on) high
        const uint32_t w = codes | (__shfl_xor_sync(0xffffffffu, codes, 4) << 4);
        if constexpr (v_has_fifth(VT)) {
#pragma unroll
            for (int off = 1; off <= 4; off <<= 1) high |= __shfl_xor_sync(0xffffffffu, high, off);
        }
        if (write) {
            if (i < 4) *reinterpret_cast<uint32_t*>(ph + G::kOffVq + t * 64 + b * 16 + 4 * i) = w;
            if (i == 0) {
                *reinterpret_cast<__half*>(ph + G::kOffVd + t * 8 + 2 * b) = __float2half_rn(d);
                if constexpr (v_has_min(VT)) *reinterpret_cast<__half*>(ph + G::kOffVm + t * 8 + 2 * b) = __float2half_rn(lo);
                if constexpr (v_has_fifth(VT)) *reinterpret_cast<uint32_t*>(ph + G::kOffVh + t * 16 + 4 * b) = high;
            }
        }
    }
}

// ----------------------------------------------------------------------------
// Append.  CTA = (row, group of its heads): the rotation's 64 angles of a row
// are computed once per CTA, in fp64 (a position of 10^6 leaves an fp32 angle
// 0.06 rad off, and a K code decided next to a border has to come out as the
// formula's), then each warp takes heads in turn: K and V of a kv head, then Q
// heads.  The rotation itself runs in fp64 too: two operations and three
// conversions a value.
// What bounds it: latency.  A row is one chain (sequence, angles, page, then its
// values); 9,022 rows, 32 / 8 heads, take 107 us (31 for their bytes), with issue
// slots at 55 % and most stalls waits for loads and at the block's two barriers.
// ----------------------------------------------------------------------------
constexpr int kAppendWarps = 8;

template <int VT, int KT, int DT>
__global__ void __launch_bounds__(kAppendWarps * 32) append_pages_kernel(const AppendPagesArgs a, int heads_per_cta) {
    using G = PageGeom<VT, KT>;
    __shared__ double2 cs[64];
    __shared__ int sSeqPos[2];
    const int row = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (warp == 0) {
        const int i = find_seq(a.batch, row);
        int pos = 0;
        if (i >= 0) pos = a.batch.seq_len[i] - (a.batch.q_start[i + 1] - row);
        if (lane == 0) {
            sSeqPos[0] = i;
            sSeqPos[1] = pos;
        }
    }
    __syncthreads();
    const int seq = sSeqPos[0], own_pos = sSeqPos[1];
    if (seq < 0) return;  // padding
    const int half = a.rot >> 1;
    if (threadIdx.x < half) {
        const double p = a.positions ? a.positions[row] : (double)own_pos + a.pos_offset;
        double s, c;
        sincos(p * (double)a.inv_freq[threadIdx.x], &s, &c);
        cs[threadIdx.x] = make_double2(c * a.mscale, s * a.mscale);
    }
    __syncthreads();

    const int n_kv = a.pool.n_kv;
    const int h0 = blockIdx.y * heads_per_cta, h1 = min(h0 + heads_per_cta, n_kv + a.n_qh);
    int page = -1;
    if (own_pos >= 0 && h0 < n_kv) {
        page = page_of(a.pool, a.batch, seq, own_pos);
        if (page < 0 && threadIdx.x == 0 && a.batch.status) atomicOr(a.batch.status, kErrBadPage);
    }
    // the lane's four dims: cosine, signed sine and the partner's dim
    double c[4], s[4];
    int partner[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const int d = 4 * lane + u;
        c[u] = 1.0;
        s[u] = 0.0;
        partner[u] = d;
        if (d < a.rot) {
            const bool second = a.interleaved ? (d & 1) : d >= half;
            const int j = a.interleaved ? d >> 1 : (second ? d - half : d);
            partner[u] = a.interleaved ? d ^ 1 : (second ? j : d + half);
            c[u] = cs[j].x;
            s[u] = second ? cs[j].y : -cs[j].y;
        }
    }
    auto rotate = [&](const float (&x)[4], double (&r)[4]) {
        float y[4];
        if (a.interleaved) {  // the lane's own other element
            y[0] = x[1]; y[1] = x[0]; y[2] = x[3]; y[3] = x[2];
        } else if ((half & 3) == 0) {  // the same element of one other lane
#pragma unroll
            for (int u = 0; u < 4; ++u) y[u] = __shfl_sync(0xffffffffu, x[u], partner[0] >> 2);
        } else {
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                // lane partner/4, element partner%4: the same for no two elements in
                // general, so all four are fetched and one picked
                const int from = partner[u] >> 2, el = partner[u] & 3;
                float v[4];
#pragma unroll
                for (int w = 0; w < 4; ++w) v[w] = __shfl_sync(0xffffffffu, x[w], from);
                y[u] = el == 0 ? v[0] : (el == 1 ? v[1] : (el == 2 ? v[2] : v[3]));
            }
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) r[u] = 4 * lane + u < a.rot ? c[u] * (double)x[u] + s[u] * (double)y[u] : (double)x[u];
    };
#pragma unroll 2
    for (int h = h0 + warp; h < h1; h += kAppendWarps) {
        float x[4];
        if (h < n_kv) {
            float v[4];
            load4<DT>(a.k.p, row * a.k.row + h * a.k.head + 4 * lane, x);
            load4<DT>(a.v.p, row * a.v.row + h * a.v.head + 4 * lane, v);
            if (a.rot) {  // uniform
                double r[4];
                rotate(x, r);
#pragma unroll
                for (int u = 0; u < 4; ++u) x[u] = (float)r[u];
            }
            uint8_t* ph = a.pool.pages + ((size_t)max(page, 0) * n_kv + h) * G::kHeadBytes;
            store_kv<VT, KT>(ph, own_pos & 255, x, v, page >= 0);
        } else {
            const int qh = h - n_kv;
            load4<DT>(a.q.p, row * a.q.row + qh * a.q.head + 4 * lane, x);
            const long long to = row * a.q_out.row + qh * a.q_out.head + 4 * lane;
            if (a.rot) {
                double r[4];
                rotate(x, r);
                store4<DT>(a.q_out.p, to, r);
            } else store4<DT>(a.q_out.p, to, x);
        }
    }
}

// ----------------------------------------------------------------------------
// Read-back: a warp per (row, kv head), lane = values 4 lane .. 4 lane + 3.
// ----------------------------------------------------------------------------
template <int VT, int KT>
__device__ __forceinline__ void read_k(const uint8_t* ph, int t, float (&x)[4]) {
    using G = PageGeom<VT, KT>;
    const int lane = threadIdx.x & 31;
    if constexpr (KT == kKF16) {
        load4<kDtF16>(ph, t * 128 + 4 * lane, x);
    } else {
        const uint32_t w = *reinterpret_cast<const uint32_t*>(ph + t * G::kKqRow + 4 * lane);
        const float d = __half2float(*reinterpret_cast<const __half*>(ph + G::kOffKd + t * 8 + 2 * (lane >> 3)));
#pragma unroll
        for (int u = 0; u < 4; ++u) x[u] = d * static_cast<float>(static_cast<int8_t>(w >> (8 * u)));
    }
}
template <int VT, int KT>
__device__ __forceinline__ void read_v(const uint8_t* ph, int t, float (&x)[4]) {
    using G = PageGeom<VT, KT>;
    const int lane = threadIdx.x & 31, b = lane >> 3, i = lane & 7;
    if constexpr (VT == kVF16) {
        load4<kDtF16>(ph + G::kOffVq, t * 128 + 4 * lane, x);
        return;
    } else {
        const float d = __half2float(*reinterpret_cast<const __half*>(ph + G::kOffVd + t * 8 + 2 * b));
        if constexpr (VT == kVQ8_0) {
            const uint32_t w = *reinterpret_cast<const uint32_t*>(ph + G::kOffVq + t * G::kVqRow + 4 * lane);
#pragma unroll
            for (int u = 0; u < 4; ++u) x[u] = d * static_cast<float>(static_cast<int8_t>(w >> (8 * u)));
        } else {
            uint32_t w = *reinterpret_cast<const uint32_t*>(ph + G::kOffVq + t * 64 + b * 16 + 4 * (i & 3));
            w = (w >> (i & 4)) & 0x0f0f0f0fu;
            uint32_t high = 0;
            if constexpr (v_has_fifth(VT)) high = *reinterpret_cast<const uint32_t*>(ph + G::kOffVh + t * 16 + 4 * b) >> (4 * i);
            float m = 0.0f;
            if constexpr (v_has_min(VT)) m = __half2float(*reinterpret_cast<const __half*>(ph + G::kOffVm + t * 8 + 2 * b));
            constexpr int kZero = v_has_min(VT) ? 0 : (VT == kVQ5_0 ? 16 : 8);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int q = static_cast<int>((w >> (8 * u)) & 15u) + static_cast<int>(((high >> u) & 1u) << 4) - kZero;
                x[u] = fmaf(d, static_cast<float>(q), m);  // d q is exact in fp32
            }
        }
    }
}

constexpr int kReadWarps = 8;

template <int VT, int KT, int DT>
__global__ void __launch_bounds__(kReadWarps * 32) read_pages_kernel(const ReadPagesArgs a) {
    using G = PageGeom<VT, KT>;
    const int row = blockIdx.x * kReadWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (row >= a.batch.n_rows) return;
    const int seq = find_seq(a.batch, row);
    if (seq < 0) return;  // padding
    const int pos = a.batch.seq_len[seq] - (a.batch.q_start[seq + 1] - row);
    int page = -1;
    if (pos >= 0) {
        page = page_of(a.pool, a.batch, seq, pos);
        if (page < 0 && lane == 0 && a.batch.status) atomicOr(a.batch.status, kErrBadPage);
    }
    const float none = pos < 0 ? 0.0f : __int_as_float(0x7fffffff);
    const int t = pos & 255;
#pragma unroll 2
    for (int h = 0; h < a.pool.n_kv; ++h) {
        const uint8_t* ph = a.pool.pages + ((size_t)max(page, 0) * a.pool.n_kv + h) * G::kHeadBytes;
        float k[4] = {none, none, none, none}, v[4] = {none, none, none, none};
        if (page >= 0) {
            if (a.k.p) read_k<VT, KT>(ph, t, k);
            if (a.v.p) read_v<VT, KT>(ph, t, v);
        }
        if (a.k.p) store4<DT>(a.k.p, row * a.k.row + h * a.k.head + 4 * lane, k);
        if (a.v.p) store4<DT>(a.v.p, row * a.v.row + h * a.v.head + 4 * lane, v);
    }
}

// calls f with the K/V pair and the value type as compile-time constants
template <class F>
cudaError_t by_types(int k_type, int v_type, int dtype, F f) {
    auto by_dtype = [&](auto vt, auto kt) {
        switch (dtype) {
            case kDtF16: return f(vt, kt, std::integral_constant<int, kDtF16>{});
            case kDtBF16: return f(vt, kt, std::integral_constant<int, kDtBF16>{});
            default: return f(vt, kt, std::integral_constant<int, kDtF32>{});
        }
    };
    std::integral_constant<int, kKQ8_0> q8;
    if (k_type == kKF16) return by_dtype(std::integral_constant<int, kVF16>{}, std::integral_constant<int, kKF16>{});
    switch (v_type) {
        case kVF16: return by_dtype(std::integral_constant<int, kVF16>{}, q8);
        case kVQ4_1: return by_dtype(std::integral_constant<int, kVQ4_1>{}, q8);
        case kVQ5_0: return by_dtype(std::integral_constant<int, kVQ5_0>{}, q8);
        case kVQ5_1: return by_dtype(std::integral_constant<int, kVQ5_1>{}, q8);
        case kVQ8_0: return by_dtype(std::integral_constant<int, kVQ8_0>{}, q8);
        default: return by_dtype(std::integral_constant<int, kVQ4_0>{}, q8);
    }
}

}  // namespace

cudaError_t launch_append_pages(const AppendPagesArgs& a, int dtype, int n_sms, cudaStream_t s) {
    const int heads = a.pool.n_kv + a.n_qh;
    // few rows: one head a warp, so that a step's latency is one head's; many
    // rows: a CTA takes all heads of its row and computes the angles once
    const int per = a.batch.n_rows * ((heads + kAppendWarps - 1) / kAppendWarps) <= 4 * n_sms ? kAppendWarps : heads;
    const dim3 grid(a.batch.n_rows, (heads + per - 1) / per);
    return by_types(a.pool.k_type, a.pool.v_type, dtype, [&](auto vt, auto kt, auto dt) {
        append_pages_kernel<vt(), kt(), dt()><<<grid, kAppendWarps * 32, 0, s>>>(a, per);
        return cudaGetLastError();
    });
}

cudaError_t launch_read_pages(const ReadPagesArgs& a, int dtype, int n_sms, cudaStream_t s) {
    (void)n_sms;
    const int grid = (a.batch.n_rows + kReadWarps - 1) / kReadWarps;
    return by_types(a.pool.k_type, a.pool.v_type, dtype, [&](auto vt, auto kt, auto dt) {
        read_pages_kernel<vt(), kt(), dt()><<<grid, kReadWarps * 32, 0, s>>>(a);
        return cudaGetLastError();
    });
}

}  // namespace kvs
