// kvs_pages.cpp -- host entry points of the batch operators over caller-owned
// pages: argument checks, tensor maps, workspace layout, launches.  Nothing
// here allocates or synchronizes.
#include <cmath>
#include <cstdio>
#include <mutex>

#include "../../include/kvs.h"
#include "kvs_pages.h"

using namespace kvs;

namespace {

int fail(int code, const char* msg) {
    set_last_error(msg);  // read back with kvs_last_error(NULL)
    return code;
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                  const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encoder() {
    static std::mutex mu;
    static EncodeTiledFn fn = nullptr;
    std::lock_guard<std::mutex> lock(mu);
    if (!fn) {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult qr;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &qr) == cudaSuccess &&
            qr == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(p);
    }
    return fn;
}

// K or V codes of all page heads as boxes of 128 tokens.  Rows of 64 bytes (4-
// and 5-bit codes) take the 64-byte swizzle, rows of 128 bytes the 128-byte
// one; fp16 rows are two 128-byte halves.  Page heads are a dimension of their
// own, so no coordinate grows with the pool's bytes.
bool encode(CUtensorMap* map, const PagePool& p, int row_bytes) {
    const cuuint64_t head_bytes = (cuuint64_t)page_head_bytes(p.v_type, p.k_type), heads = (cuuint64_t)p.n_pages * p.n_kv;
    const EncodeTiledFn fn = encoder();
    if (!fn) return false;
    const cuuint32_t ones[4] = {1, 1, 1, 1};
    if (row_bytes == 256) {
        const cuuint64_t dims[4] = {128, 2, head_bytes / 256, heads}, strides[3] = {128, 256, head_bytes};
        const cuuint32_t box[4] = {128, 1, 128, 1};
        return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, p.pages, dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
    }
    const cuuint64_t w = (cuuint64_t)row_bytes;
    const cuuint64_t dims[3] = {w, head_bytes / w, heads}, strides[2] = {w, head_bytes};
    const cuuint32_t box[3] = {(cuuint32_t)row_bytes, 128, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, p.pages, dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
              row_bytes == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Launches go to the device that owns the pool; the caller's current device is
// put back at the end.
struct OnDevice {
    int before = -1, dev = -1;
    int enter(const void* p) {
        cudaPointerAttributes at;
        if (cudaPointerGetAttributes(&at, p) != cudaSuccess) {
            cudaGetLastError();
            return fail(KVS_E_CUDA, "no usable CUDA device");
        }
        if (at.type != cudaMemoryTypeDevice && at.type != cudaMemoryTypeManaged)
            return fail(KVS_E_INVAL, "pool pages must be device memory");
        dev = at.device;
        if (cudaGetDevice(&before) != cudaSuccess) return fail(KVS_E_CUDA, "cudaGetDevice failed");
        if (before != dev && cudaSetDevice(dev) != cudaSuccess) return fail(KVS_E_CUDA, "cudaSetDevice failed");
        return KVS_OK;
    }
    ~OnDevice() {
        if (before >= 0 && before != dev) cudaSetDevice(before);
    }
    int n_sms() const {
        int n = 0;
        cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
        return n > 0 ? n : 1;
    }
};

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
int dtype_bytes(int dtype) { return dtype == KVS_DT_F32 ? 4 : 2; }

int check_pool(const kvs_page_pool* p, PagePool* out) {
    if (!p || !p->pages) return fail(KVS_E_INVAL, "null pool or pages");
    if (!kv_pair_supported(p->type_k, p->type_v)) return fail(KVS_E_INVAL, "unsupported K/V type pair");
    if (p->n_pages < 1 || p->n_kv_heads < 1) return fail(KVS_E_INVAL, "a pool has at least one page and one kv head");
    if ((long long)p->n_pages * p->n_kv_heads > 0x7fffffffll) return fail(KVS_E_INVAL, "more than 2^31 - 1 page heads in a pool");
    if (!aligned(p->pages, 16)) return fail(KVS_E_INVAL, "pages must be 16-byte aligned");
    *out = PagePool{static_cast<uint8_t*>(p->pages), p->n_pages, p->n_kv_heads, p->type_k, p->type_v};
    return KVS_OK;
}

int check_batch(const kvs_page_batch* b, PageBatch* out) {
    if (!b) return fail(KVS_E_INVAL, "null batch");
    if (b->n_seqs < 0 || b->n_rows < 0 || b->table_stride < 0 || b->max_new < 0) return fail(KVS_E_INVAL, "negative batch sizes");
    if (b->n_seqs > 0 && (!b->q_start || !b->seq_len)) return fail(KVS_E_INVAL, "null q_start or seq_len");
    if (b->n_seqs > 0 && b->table_stride > 0 && !b->page_table) return fail(KVS_E_INVAL, "null page_table");
    if (!aligned(b->q_start, 4) || !aligned(b->seq_len, 4) || !aligned(b->page_table, 4) || !aligned(b->status, 4))
        return fail(KVS_E_INVAL, "batch arrays must be 4-byte aligned");
    *out = PageBatch{b->n_seqs, b->n_rows, b->q_start, b->seq_len, b->page_table, b->table_stride, b->status};
    return KVS_OK;
}

bool dtype_ok(int d) { return d == KVS_DT_F16 || d == KVS_DT_BF16 || d == KVS_DT_F32; }

// n_rows: of the batch; a tensor of no rows may have a null address
int check_rows(const kvs_page_rows* r, int dtype, int n_rows, const char* what, RowsRef* out) {
    static thread_local char msg[128];
    if (!r || (!r->data && n_rows > 0)) {
        snprintf(msg, sizeof msg, "null %s", what);
        return fail(KVS_E_INVAL, msg);
    }
    const long long unit = 16 / dtype_bytes(dtype);
    if (!aligned(r->data, 16) || r->row_stride % unit || r->head_stride % unit) {
        snprintf(msg, sizeof msg, "%s: address and strides must be multiples of 16 bytes", what);
        return fail(KVS_E_INVAL, msg);
    }
    *out = RowsRef{r->data, r->row_stride, r->head_stride};
    return KVS_OK;
}

int launched(cudaError_t e) { return e == cudaSuccess ? KVS_OK : fail(KVS_E_CUDA, cudaGetErrorString(e)); }

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

// the workspace: arrival counters, the many-row kernel's plan, records of shared
// units (both kernels' in turn), the prefix's records
struct Workspace {
    size_t counters = 0, plan, units, records, prior_acc, prior_ml, bytes;
    Workspace(long long n_rows, long long n_seqs, long long n_qh, int group) {
        const bool wide = n_rows * group > kFewSeqRows;
        plan = up256((size_t)kFewCtas * sizeof(int));
        units = plan + up256(sizeof(WidePlan));
        records = units + (wide ? up256((size_t)wide_groups(n_rows, group, n_seqs) * sizeof(WideUnit)) : 0);
        prior_acc = records + up256(wide && kWideRecordBytes > kFewRecordBytes ? kWideRecordBytes : kFewRecordBytes);
        prior_ml = prior_acc + up256((size_t)n_rows * n_qh * kHeadDim * sizeof(float));
        bytes = prior_ml + up256((size_t)n_rows * n_qh * sizeof(float2));
    }
};

}  // namespace

extern "C" int kvs_append_pages(const kvs_page_pool* pool, const kvs_page_batch* batch, int dtype, const kvs_page_rows* k,
                                const kvs_page_rows* v, int n_q_heads, const kvs_page_rows* q, const kvs_page_rows* q_out,
                                const kvs_rope* rope, void* stream) {
    AppendPagesArgs a{};
    int rc = check_pool(pool, &a.pool);
    if (rc == KVS_OK) rc = check_batch(batch, &a.batch);
    if (rc != KVS_OK) return rc;
    if (!dtype_ok(dtype)) return fail(KVS_E_INVAL, "unknown dtype");
    if ((rc = check_rows(k, dtype, batch->n_rows, "k", &a.k)) != KVS_OK || (rc = check_rows(v, dtype, batch->n_rows, "v", &a.v)) != KVS_OK) return rc;
    if ((q == nullptr) != (q_out == nullptr)) return fail(KVS_E_INVAL, "q and q_out go together");
    if (q) {
        if (n_q_heads < 1) return fail(KVS_E_INVAL, "n_q_heads must be positive when q is given");
        if ((rc = check_rows(q, dtype, batch->n_rows, "q", &a.q)) != KVS_OK || (rc = check_rows(q_out, dtype, batch->n_rows, "q_out", &a.q_out)) != KVS_OK) return rc;
        a.n_qh = n_q_heads;
    }
    if ((long long)a.pool.n_kv + a.n_qh > 65535) return fail(KVS_E_INVAL, "more than 65535 heads");
    if (rope && rope->rot_dim != 0) {
        if (rope->rot_dim < 0 || rope->rot_dim > kHeadDim || rope->rot_dim % 2) return fail(KVS_E_INVAL, "rot_dim must be even, 0..128");
        if (!rope->inv_freq || !aligned(rope->inv_freq, 4) || !aligned(rope->positions, 4))
            return fail(KVS_E_INVAL, "rope: null inv_freq, or an array not 4-byte aligned");
        if (!std::isfinite(rope->mscale)) return fail(KVS_E_INVAL, "rope: mscale must be finite");
        a.inv_freq = rope->inv_freq;
        a.rot = rope->rot_dim;
        a.interleaved = rope->interleaved != 0;
        a.positions = rope->positions;
        a.pos_offset = rope->pos_offset;
        a.mscale = rope->mscale == 0.0f ? 1.0f : rope->mscale;
    }
    OnDevice on;
    if ((rc = on.enter(pool->pages)) != KVS_OK) return rc;
    if (a.batch.n_rows == 0 || a.batch.n_seqs == 0) return KVS_OK;
    return launched(launch_append_pages(a, dtype, on.n_sms(), static_cast<cudaStream_t>(stream)));
}

extern "C" int kvs_read_pages(const kvs_page_pool* pool, const kvs_page_batch* batch, int dtype, const kvs_page_rows* k,
                              const kvs_page_rows* v, void* stream) {
    ReadPagesArgs a{};
    int rc = check_pool(pool, &a.pool);
    if (rc == KVS_OK) rc = check_batch(batch, &a.batch);
    if (rc != KVS_OK) return rc;
    if (!dtype_ok(dtype)) return fail(KVS_E_INVAL, "unknown dtype");
    if (!k && !v) return fail(KVS_E_INVAL, "neither k nor v is wanted");
    if (k && (rc = check_rows(k, dtype, batch->n_rows, "k", &a.k)) != KVS_OK) return rc;
    if (v && (rc = check_rows(v, dtype, batch->n_rows, "v", &a.v)) != KVS_OK) return rc;
    OnDevice on;
    if ((rc = on.enter(pool->pages)) != KVS_OK) return rc;
    if (a.batch.n_rows == 0 || a.batch.n_seqs == 0) return KVS_OK;
    return launched(launch_read_pages(a, dtype, on.n_sms(), static_cast<cudaStream_t>(stream)));
}

extern "C" size_t kvs_attend_pages_workspace(const kvs_page_batch* batch, int n_q_heads, int n_kv_heads) {
    if (!batch || batch->n_rows < 0 || batch->n_seqs < 0 || n_kv_heads < 1 || n_q_heads < 1 || n_q_heads % n_kv_heads) {
        set_last_error("kvs_attend_pages_workspace: bad argument");
        return 0;
    }
    return Workspace(batch->n_rows, batch->n_seqs, n_q_heads, n_q_heads / n_kv_heads).bytes;
}

extern "C" int kvs_attend_pages(const kvs_page_pool* pool, const kvs_page_batch* batch, int q_dtype, int n_q_heads,
                                const kvs_page_rows* q, int out_dtype, const kvs_page_rows* out, float* lse,
                                const kvs_score* score, const kvs_page_prefix* prefix, void* workspace, size_t workspace_bytes,
                                void* stream) {
    AttendPagesArgs a{};
    int rc = check_pool(pool, &a.pool);
    if (rc == KVS_OK) rc = check_batch(batch, &a.batch);
    if (rc != KVS_OK) return rc;
    if (n_q_heads < 1 || n_q_heads % a.pool.n_kv) return fail(KVS_E_INVAL, "n_q_heads must be a positive multiple of n_kv_heads");
    if (q_dtype != KVS_DT_F16 && q_dtype != KVS_DT_BF16) return fail(KVS_E_INVAL, "q is F16 or BF16");
    if (!dtype_ok(out_dtype)) return fail(KVS_E_INVAL, "unknown out_dtype");
    if ((rc = check_rows(q, q_dtype, batch->n_rows, "q", &a.q)) != KVS_OK || (rc = check_rows(out, out_dtype, batch->n_rows, "out", &a.out)) != KVS_OK) return rc;
    if (!aligned(lse, 4)) return fail(KVS_E_INVAL, "lse must be 4-byte aligned");
    a.n_qh = n_q_heads;
    a.group = n_q_heads / a.pool.n_kv;
    if ((long long)a.batch.n_rows * a.group > 0x7fffffffll) return fail(KVS_E_INVAL, "more than 2^31 - 1 rows per kv head");
    a.q_dtype = q_dtype;
    a.out_dtype = out_dtype;
    a.precise = out_dtype != KVS_DT_BF16;
    a.lse = lse;
    a.scale = 0.08838834764831845f;  // 1/sqrt(128)
    if (score) {
        if (!std::isfinite(score->scale) || !std::isfinite(score->softcap) || score->softcap < 0.0f || score->window < 0 ||
            (score->softcap > 0.0f && !std::isfinite(1.0f / score->softcap)))
            return fail(KVS_E_INVAL, "score: scale and softcap must be finite, softcap and window not negative");
        if (!aligned(score->alibi_slopes, 4) || !aligned(score->first_key, 4) || !aligned(score->end_key, 4))
            return fail(KVS_E_INVAL, "score arrays must be 4-byte aligned");
        if (score->scale != 0.0f) a.scale = score->scale;
        a.softcap = score->softcap;
        a.inv_cap = a.softcap > 0.0f ? 1.0f / a.softcap : 0.0f;
        a.window = score->window;
        a.slopes = score->alibi_slopes;
        a.first_key = score->first_key;
        a.end_key = score->end_key;
    }
    if (prefix && prefix->n_tokens != 0) {
        if (prefix->n_tokens < 0 || !prefix->page_table || !aligned(prefix->page_table, 4))
            return fail(KVS_E_INVAL, "prefix: negative length, or a null or misaligned page_table");
        a.prefix_table = prefix->page_table;
        a.prefix_len = prefix->n_tokens;
    }
    const Workspace w(a.batch.n_rows, a.batch.n_seqs, n_q_heads, a.group);
    if (!workspace || !aligned(workspace, 256) || workspace_bytes < w.bytes)
        return fail(KVS_E_INVAL, "workspace: null, not 256-byte aligned, or smaller than kvs_attend_pages_workspace says");
    uint8_t* base = static_cast<uint8_t*>(workspace);
    a.counters = reinterpret_cast<int*>(base + w.counters);
    a.plan = reinterpret_cast<WidePlan*>(base + w.plan);
    a.units = reinterpret_cast<WideUnit*>(base + w.units);
    a.records = reinterpret_cast<float*>(base + w.records);
    a.prior_acc = reinterpret_cast<float*>(base + w.prior_acc);
    a.prior_ml = reinterpret_cast<float2*>(base + w.prior_ml);
    OnDevice on;
    if ((rc = on.enter(pool->pages)) != KVS_OK) return rc;
    if (a.batch.n_rows == 0 || a.batch.n_seqs == 0) return KVS_OK;

    PageMaps maps;
    const int v_row = a.pool.v_type == kVF16 ? 256 : (a.pool.v_type == kVQ8_0 ? 128 : 64);
    if (!encode(&maps.k, a.pool, a.pool.k_type == kKF16 ? 256 : 128) || !encode(&maps.v, a.pool, v_row))
        return fail(KVS_E_CUDA, "cuTensorMapEncodeTiled failed");
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int n_sms = on.n_sms();
    // Up to 32 rows per kv head go to the few-row kernel (HBM bound, fp32-class
    // sums), more to the tensor-core kernel.
    auto few = [&](AttendPagesArgs& x, long long rows) {
        return launched(launch_attend_few(x, maps, rows <= 8 ? 8 : kFewRowsMax, n_sms, s));
    };
    const long long all = (long long)a.batch.n_rows * a.group;
    if (a.prefix_len > 0) {
        AttendPagesArgs p = a;
        p.prefix_phase = 1;
        rc = all > kFewSeqRows ? launched(launch_attend_wide(p, maps, n_sms, s)) : few(p, all);
        if (rc != KVS_OK) return rc;
    }
    const long long most = (batch->max_new > 0 && batch->max_new < a.batch.n_rows ? batch->max_new : a.batch.n_rows) * (long long)a.group;
    if (most <= kFewSeqRows) {
        a.few_rows = 0x7fffffff;
        return few(a, most);
    }
    // Each kernel takes its sequences by their rows on the device: single tokens
    // beside prompts, or a short sequence in tensors made for more.  One sequence
    // whose rows the caller states needs no second launch (8 to 11 us behind a
    // 256-token chunk or packed documents).
    a.few_rows = a.batch.n_seqs == 1 && batch->max_new > 0 ? 0 : kFewSeqRows;
    rc = launched(launch_attend_wide(a, maps, n_sms, s));
    return rc == KVS_OK && a.few_rows > 0 ? few(a, a.group) : rc;
}
