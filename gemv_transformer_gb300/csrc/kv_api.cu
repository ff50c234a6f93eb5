// kv_api.cu -- entry points of the rotary and paged-cache calls (declared in include/wq.h):
// argument checks and launches, nothing else.
#include <cmath>

#include "kv_internal.h"

namespace wq {
namespace {

constexpr int kMaxHeadDim = 256;
constexpr long long kMaxSlots = 1ll << 30;  // a slot number and a tile beyond it fit an int

bool aligned(const void *p, uintptr_t to) { return ((uintptr_t)p & (to - 1)) == 0; }
wq_status cuda_status(cudaError_t e) { return e == cudaSuccess ? WQ_OK : WQ_ERR_CUDA; }
int element_bytes(int dtype) { return dtype == WQ_F32 ? 4 : 2; }

// The cache's restrictions; fills the kernels' view of it.
bool view_of(const wq_kv_cache *c, int n_seq, const int32_t *page_table, int max_pages,
             KvView &out) {
    if (!c || n_seq <= 0 || max_pages <= 0) return false;
    if (c->dtype != WQ_BF16 && c->dtype != WQ_F16 && c->dtype != WQ_F32) return false;
    if (c->n_pages <= 0 || c->page_size <= 0 || c->n_heads <= 0 || c->head_dim <= 0) return false;
    if (c->head_dim % 8 || c->head_dim > kMaxHeadDim) return false;
    if (!c->k || !c->v || !aligned(c->k, 16) || !aligned(c->v, 16)) return false;
    if ((long long)max_pages * c->page_size > kMaxSlots) return false;
    const int eb = element_bytes(c->dtype);
    const int64_t strides[3] = {c->page_stride, c->head_stride, c->token_stride};
    const int extents[3] = {c->n_pages, c->n_heads, c->page_size};
    for (int i = 0; i < 3; ++i) {
        if (strides[i] < c->head_dim || strides[i] > INT64_MAX / 64) return false;
        if ((strides[i] * eb) % 16) return false;
        if (strides[i] > INT64_MAX / 64 / extents[i]) return false;  // offsets fit 64 bits
    }
    out.k = static_cast<char *>(c->k);
    out.v = static_cast<char *>(c->v);
    out.page_stride = c->page_stride * eb;
    out.head_stride = c->head_stride * eb;
    out.token_stride = c->token_stride * eb;
    out.page_size = make_fast_div((uint32_t)c->page_size);
    out.n_pages = c->n_pages;
    out.max_pages = max_pages;
    out.n_heads = c->n_heads;
    out.head_dim = c->head_dim;
    out.dtype = c->dtype;
    out.page_table = page_table;
    return true;
}

bool rope_ok(int head_dim, int rot, unsigned flags, const int32_t *pos, const float *table,
             int table_rows) {
    if (head_dim <= 0 || head_dim > kMaxHeadDim || rot < 0 || rot > head_dim || rot % 2)
        return false;
    if (flags & ~(unsigned)(WQ_ROPE_INTERLEAVED | WQ_ROPE_TRANSPOSE)) return false;
    return rot == 0 || (pos && table && aligned(table, 16) && table_rows > 0);
}

// Rows of n_heads heads at x + t * stride.
bool rows_ok(const float *x, int64_t stride, int n_heads, int head_dim) {
    return x && aligned(x, 4) && stride >= (int64_t)n_heads * head_dim &&
           stride <= INT64_MAX / 64 / 0x7FFFFFFF;
}

bool workspace_ok(const void *workspace, size_t bytes, size_t need) {
    return need == 0 || (workspace && aligned(workspace, 256) && bytes >= need);
}

RopeArgs rope_args(int head_dim, int rot, unsigned flags, const int32_t *pos, const float *table,
                   int table_rows, const DeviceInfo &dev) {
    return {head_dim, rot, flags, pos, reinterpret_cast<const float2 *>(table), table_rows,
            dev.status};
}

int cut(int n, long long to) { return to < n ? (int)to : n; }

}  // namespace
}  // namespace wq

using namespace wq;

extern "C" {

wq_status wq_rope_table(int rows, int rot, double base, const wq_rope_scaling *scaling,
                        float *table, wq_stream_t stream) {
    if (rows <= 0 || rot <= 0 || rot % 2 || rot > kMaxHeadDim) return WQ_ERR_INVALID_ARG;
    if (!(base > 1.0) || !std::isfinite(base)) return WQ_ERR_INVALID_ARG;
    if (!table || !aligned(table, 16)) return WQ_ERR_INVALID_ARG;
    wq_rope_scaling sc{};
    if (scaling) sc = *scaling;
    if (sc.kind < WQ_ROPE_PLAIN || sc.kind > WQ_ROPE_BANDS) return WQ_ERR_INVALID_ARG;
    if (!std::isfinite(sc.magnitude) || sc.magnitude < 0.0) return WQ_ERR_INVALID_ARG;
    if (sc.kind != WQ_ROPE_PLAIN && (!(sc.factor > 0.0) || !std::isfinite(sc.factor)))
        return WQ_ERR_INVALID_ARG;
    if (sc.kind == WQ_ROPE_NTK &&
        (rot < 4 || !std::isfinite(base * std::pow(sc.factor, (double)rot / (rot - 2)))))
        return WQ_ERR_INVALID_ARG;
    if (sc.kind == WQ_ROPE_YARN || sc.kind == WQ_ROPE_BANDS) {
        if (sc.original <= 0 || !(sc.low > 0.0) || !(sc.high > sc.low) || !std::isfinite(sc.high))
            return WQ_ERR_INVALID_ARG;
    }
    if (sc.magnitude == 0.0)
        sc.magnitude =
            sc.kind == WQ_ROPE_YARN && sc.factor > 1.0 ? 0.1 * std::log(sc.factor) + 1.0 : 1.0;
    DeviceInfo dev;
    if (!device_info(dev)) return WQ_ERR_CUDA;
    return cuda_status(launch_rope_table(rows, rot, base, sc, table, dev, (cudaStream_t)stream));
}

wq_status wq_rope(int n, int n_heads, int head_dim, int rot, unsigned flags, const float *x,
                  int64_t x_stride, const int32_t *pos, const float *table, int table_rows,
                  float *out, int64_t out_stride, wq_stream_t stream) {
    if (n <= 0 || n_heads <= 0 || !rope_ok(head_dim, rot, flags, pos, table, table_rows))
        return WQ_ERR_INVALID_ARG;
    if (!rows_ok(x, x_stride, n_heads, head_dim) || !rows_ok(out, out_stride, n_heads, head_dim))
        return WQ_ERR_INVALID_ARG;
    if (out == x && out_stride != x_stride) return WQ_ERR_INVALID_ARG;
    DeviceInfo dev;
    if (!device_info(dev)) return WQ_ERR_CUDA;
    return cuda_status(launch_rope(rope_args(head_dim, rot, flags, pos, table, table_rows, dev), x,
                                   x_stride, n, n_heads, out, out_stride, dev,
                                   (cudaStream_t)stream));
}

wq_status wq_kv_append(const wq_kv_cache *cache, int n_tok, int h_q, int rot, unsigned flags,
                       const float *q, int64_t q_stride, const float *k, int64_t k_stride,
                       const float *v, int64_t v_stride, const int32_t *pos, const float *table,
                       int table_rows, int n_seq, const int32_t *seq, const int32_t *slot,
                       const int32_t *page_table, int max_pages, float *q_out,
                       int64_t q_out_stride, float *acc, int32_t *slot_pos, int64_t acc_stride,
                       wq_stream_t stream) {
    KvView kv;
    if (!view_of(cache, n_seq, page_table, max_pages, kv)) return WQ_ERR_INVALID_ARG;
    if (n_tok <= 0 || h_q < 0 || !page_table || !slot || (!seq && n_seq < n_tok))
        return WQ_ERR_INVALID_ARG;
    if (!rope_ok(kv.head_dim, rot, flags, pos, table, table_rows)) return WQ_ERR_INVALID_ARG;
    if (!rows_ok(k, k_stride, kv.n_heads, kv.head_dim) ||
        !rows_ok(v, v_stride, kv.n_heads, kv.head_dim))
        return WQ_ERR_INVALID_ARG;
    if (h_q > 0 && (!rows_ok(q, q_stride, h_q, kv.head_dim) ||
                    !rows_ok(q_out, q_out_stride, h_q, kv.head_dim) ||
                    (q_out == q && q_out_stride != q_stride)))
        return WQ_ERR_INVALID_ARG;
    if ((acc || slot_pos) && acc_stride < 1) return WQ_ERR_INVALID_ARG;
    if (slot_pos && !pos) return WQ_ERR_INVALID_ARG;
    DeviceInfo dev;
    if (!device_info(dev)) return WQ_ERR_CUDA;
    AppendArgs a{};
    a.rope = rope_args(kv.head_dim, rot, flags, pos, table, table_rows, dev);
    a.n_tok = n_tok;
    a.h_q = h_q;
    a.n_seq = n_seq;
    a.n_slots = max_pages * (int)kv.page_size.d;
    if (acc || slot_pos) a.n_slots = cut(a.n_slots, acc_stride);
    a.q = q;
    a.k = k;
    a.v = v;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.q_out = q_out;
    a.q_out_stride = q_out_stride;
    a.seq = seq;
    a.slot = slot;
    a.acc = acc;
    a.slot_pos = slot_pos;
    a.acc_stride = acc_stride;
    return cuda_status(launch_kv_append(a, kv, dev, (cudaStream_t)stream));
}

size_t wq_attn_paged_workspace_bytes(const wq_kv_cache *cache, int n_seq, int h_q, int max_pages,
                                     int with_acc) {
    KvView kv;
    if (!view_of(cache, n_seq, nullptr, max_pages, kv) || h_q <= 0 || h_q % kv.n_heads) return 0;
    return attn_workspace_bytes(kv, n_seq, h_q, max_pages * (int)kv.page_size.d, with_acc != 0);
}

wq_status wq_attn_paged(const wq_kv_cache *cache, int n_seq, int h_q, float scale, int window,
                        const float *q, int64_t q_stride, const int32_t *page_table, int max_pages,
                        const int32_t *lens, const float *mask, int64_t mask_stride, float *out,
                        int64_t out_stride, float *lse, const float *acc_in, float *acc_out,
                        int64_t acc_stride, void *workspace, size_t workspace_bytes,
                        wq_stream_t stream) {
    KvView kv;
    if (!view_of(cache, n_seq, page_table, max_pages, kv)) return WQ_ERR_INVALID_ARG;
    if (h_q <= 0 || h_q % kv.n_heads || window < 0 || !std::isfinite(scale))
        return WQ_ERR_INVALID_ARG;
    if (!page_table || !lens) return WQ_ERR_INVALID_ARG;
    if (!rows_ok(q, q_stride, h_q, kv.head_dim) || !rows_ok(out, out_stride, h_q, kv.head_dim))
        return WQ_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(out, 16) || q_stride % 4 || out_stride % 4)
        return WQ_ERR_INVALID_ARG;
    if ((mask && mask_stride < 1) || (acc_out && acc_stride < 1) || (acc_in && !acc_out))
        return WQ_ERR_INVALID_ARG;
    const int n_slots = max_pages * (int)kv.page_size.d;
    if (!workspace_ok(workspace, workspace_bytes,
                      attn_workspace_bytes(kv, n_seq, h_q, n_slots, acc_out != nullptr)))
        return WQ_ERR_INVALID_ARG;
    DeviceInfo dev;
    if (!device_info(dev)) return WQ_ERR_CUDA;
    AttnArgs a{};
    a.n_seq = n_seq;
    a.h_q = h_q;
    a.group = h_q / kv.n_heads;
    a.n_slots = n_slots;
    if (mask) a.n_slots = cut(a.n_slots, mask_stride);
    if (acc_out) a.n_slots = cut(a.n_slots, acc_stride);
    a.scale = scale;
    a.window = window;
    a.q = q;
    a.q_stride = q_stride;
    a.lens = lens;
    a.mask = mask;
    a.mask_stride = mask_stride;
    a.out = out;
    a.out_stride = out_stride;
    a.lse = lse;
    a.acc_in = acc_in;
    a.acc_out = acc_out;
    a.acc_stride = acc_stride;
    a.workspace = workspace;
    a.status = dev.status;
    return cuda_status(launch_attn_paged(a, kv, dev, (cudaStream_t)stream));
}

size_t wq_kv_evict_workspace_bytes(const wq_kv_cache *cache, int n_seq, int max_pages, int keep) {
    KvView kv;
    if (!view_of(cache, n_seq, nullptr, max_pages, kv) || keep <= 0) return 0;
    return evict_workspace_bytes(kv, n_seq, max_pages * (int)kv.page_size.d, keep);
}

wq_status wq_kv_evict(const wq_kv_cache *cache, int n_seq, const int32_t *page_table,
                      int max_pages, const int32_t *lens, const int32_t *seen, int keep, int sinks,
                      int recent, const float *acc, const int32_t *slot_pos, float *acc_out,
                      int32_t *pos_out, int64_t acc_stride, int32_t *lens_out, void *workspace,
                      size_t workspace_bytes, wq_stream_t stream) {
    KvView kv;
    if (!view_of(cache, n_seq, page_table, max_pages, kv)) return WQ_ERR_INVALID_ARG;
    if (keep <= 0 || sinks < 0 || recent < 0 || (long long)sinks + recent > keep)
        return WQ_ERR_INVALID_ARG;
    if (!page_table || !lens || !seen || !acc || !slot_pos || !acc_out || !pos_out || !lens_out ||
        acc_stride < 1)
        return WQ_ERR_INVALID_ARG;
    const int n_slots = max_pages * (int)kv.page_size.d;
    if (!workspace_ok(workspace, workspace_bytes, evict_workspace_bytes(kv, n_seq, n_slots, keep)))
        return WQ_ERR_INVALID_ARG;
    DeviceInfo dev;
    if (!device_info(dev)) return WQ_ERR_CUDA;
    EvictArgs a{};
    a.n_seq = n_seq;
    a.n_slots = cut(n_slots, acc_stride);
    a.keep = keep;
    a.sinks = sinks;
    a.recent = recent;
    a.lens = lens;
    a.seen = seen;
    a.acc = acc;
    a.slot_pos = slot_pos;
    a.acc_out = acc_out;
    a.pos_out = pos_out;
    a.lens_out = lens_out;
    a.acc_stride = acc_stride;
    a.workspace = workspace;
    a.status = dev.status;
    return cuda_status(launch_kv_evict(a, kv, dev, (cudaStream_t)stream));
}

}  // extern "C"
