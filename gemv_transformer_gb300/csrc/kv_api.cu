// kv_api.cu -- entry points of the rotary and paged-cache calls (declared in include/wq.h):
// argument checks and launches, nothing else.
#include <cmath>

#include "kv_internal.h"

namespace wq {
namespace {

constexpr int kMaxHeadDim = 256;
constexpr long long kMaxSlots = 1ll << 30;  // a slot number and a tile beyond it fit an int
// Of attention's scale and cap, and one by it the least cap: their quotient is finite in f32, as are
// their products with log2 e.
constexpr float kMostScale = (float)(1ull << 60);
constexpr int64_t kMaxStride = INT64_MAX / 64 / 0x7FFFFFFF;  // offsets of any row fit 64 bits

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
           stride <= kMaxStride;
}

bool workspace_ok(const void *workspace, size_t bytes, size_t need) {
    return need == 0 || (workspace && aligned(workspace, 256) && bytes >= need);
}

RopeArgs rope_args(int head_dim, int rot, unsigned flags, const int32_t *pos, const float *table,
                   int table_rows, const DeviceInfo &dev) {
    return {head_dim, rot, flags, pos, reinterpret_cast<const float2 *>(table), table_rows,
            dev.status};
}

bool float_type(int type) { return type == WQ_F32 || type == WQ_BF16 || type == WQ_F16; }

bool norm_ok(const wq_head_norm *norm, NormView &out) {
    out = NormView{WQ_HEAD_NONE, 0.f, nullptr, nullptr};
    if (!norm || norm->kind == WQ_HEAD_NONE) return true;
    if (norm->kind != WQ_HEAD_RMS && norm->kind != WQ_HEAD_LAYER) return false;
    if (!std::isfinite(norm->eps) || norm->eps < 0.f) return false;
    if (!aligned(norm->weight, 4) || !aligned(norm->bias, 4)) return false;
    out = NormView{norm->kind, norm->eps, norm->weight, norm->bias};
    return true;
}

// The rotation's restrictions; fills the kernels' view of it, which pair by which axis and column.
bool axes_ok(const wq_rope_axes *r, int head_dim, AxesView &out) {
    out = AxesView{};
    if (head_dim <= 0 || head_dim > kMaxHeadDim) return false;
    if (!r || r->rot == 0) return true;
    if (r->rot < 0 || r->rot > head_dim || r->rot % 2) return false;
    const unsigned known = WQ_ROPE_INTERLEAVED | WQ_AXES_DEALT | WQ_AXES_RESTART;
    if ((r->flags & ~known) || r->axes < 1 || r->axes > 4) return false;
    if (r->table_rows <= 0 || r->table_pairs <= 0 || r->table_pairs > 128) return false;
    if (!r->pos || !r->table || !aligned(r->table, 16) || !aligned(r->pos, 4)) return false;
    if (r->axes > 1 && (r->pos_stride < 0 || r->pos_stride > INT64_MAX / 64)) return false;
    const int half = r->rot / 2;
    long long sum = 0;
    for (int a = 0; a < r->axes; ++a) {
        if (r->pairs[a] < 0 || r->pairs[a] > half) return false;
        sum += r->pairs[a];
        if ((r->flags & WQ_AXES_DEALT) && a > 0 && r->pairs[a] > 0 &&
            (r->pairs[a] - 1) * r->axes + a >= half)
            return false;
        if (r->pairs[a] > 0) out.used |= 1u << a;
    }
    if (sum != half) return false;
    int seen[4] = {0, 0, 0, 0};
    bool plain = r->table_pairs % 2 == 0;
    for (int i = 0, axis = 0, left = r->pairs[0]; i < half; ++i) {
        if (r->flags & WQ_AXES_DEALT) {
            axis = i / r->axes < r->pairs[i % r->axes] ? i % r->axes : 0;
        } else {
            while (left == 0) left = r->pairs[++axis];
            --left;
        }
        const int col = r->flags & WQ_AXES_RESTART ? seen[axis]++ : i;
        if (col >= r->table_pairs) return false;
        out.code[i] = (uint16_t)(axis << 8 | col);
        plain = plain && axis == 0 && col == i;
    }
    out.rot = r->rot;
    out.flags = r->flags & WQ_ROPE_INTERLEAVED;
    out.axes = r->axes;
    out.table_rows = r->table_rows;
    out.table_pairs = r->table_pairs;
    out.straight = plain;
    out.pos = r->pos;
    out.pos_stride = r->pos_stride;
    out.table = reinterpret_cast<const float2 *>(r->table);
    return true;
}

// Rows of n_heads heads of a 16- or 32-bit type at x + t * stride.
bool typed_rows_ok(const void *x, int type, int64_t stride, int n_heads, int head_dim) {
    return x && aligned(x, element_bytes(type)) && stride >= (int64_t)n_heads * head_dim &&
           stride <= kMaxStride;
}

int cut(int n, long long to) { return to < n ? (int)to : n; }

// wq_kv_accept; slots null: none.
wq_status accept_paths(const wq_kv_cache *caches, int n_caches, int n_seq, int n_tok,
                       const int32_t *page_table, int max_pages, const int32_t *starts,
                       const int32_t *parent, const int32_t *tokens, const int32_t *choice,
                       const int32_t *lens, int32_t *path, int32_t *accepted, int32_t *next,
                       int32_t *lens_out, const wq_slot_arrays *slots, int64_t acc_stride,
                       wq_stream_t stream) {
    if (!caches || n_caches <= 0 || n_tok <= 0) return WQ_ERR_INVALID_ARG;
    if (!page_table || !starts || !parent || !tokens || !choice || !lens || !path || !accepted ||
        !next || !lens_out || lens_out == lens)
        return WQ_ERR_INVALID_ARG;
    KvView kv, other;
    for (int i = 0; i < n_caches; ++i) {
        if (!view_of(&caches[i], n_seq, page_table, max_pages, i ? other : kv))
            return WQ_ERR_INVALID_ARG;
        const wq_kv_cache &c = caches[i], &f = caches[0];
        if (c.dtype != f.dtype || c.n_pages != f.n_pages || c.page_size != f.page_size ||
            c.n_heads != f.n_heads || c.head_dim != f.head_dim ||
            c.page_stride != f.page_stride || c.head_stride != f.head_stride ||
            c.token_stride != f.token_stride)
            return WQ_ERR_INVALID_ARG;
        if (slots && !(aligned(slots[i].acc, 4) && aligned(slots[i].slot_pos, 4)))
            return WQ_ERR_INVALID_ARG;
    }
    DeviceInfo dev;
    if (!device_info(dev)) return WQ_ERR_CUDA;
    AcceptArgs a{n_seq, n_tok, max_pages * (int)kv.page_size.d, starts, parent, tokens, choice,
                 lens, path, accepted, next, lens_out, dev.status};
    if (slots) a.n_slots = cut(a.n_slots, acc_stride);
    for (int c0 = 0; c0 < n_caches; c0 += kAcceptCaches) {
        AcceptPools pools{};
        AcceptSlots arrays{};
        arrays.stride = acc_stride;
        pools.count = n_caches - c0 < kAcceptCaches ? n_caches - c0 : kAcceptCaches;
        for (int i = 0; i < pools.count; ++i) {
            pools.k[i] = static_cast<char *>(caches[c0 + i].k);
            pools.v[i] = static_cast<char *>(caches[c0 + i].v);
            if (!slots) continue;
            arrays.p[2 * i] = slots[c0 + i].acc;
            arrays.p[2 * i + 1] = slots[c0 + i].slot_pos;
        }
        const cudaError_t err = launch_kv_accept(a, kv, pools, slots ? &arrays : nullptr, c0 == 0,
                                                 (cudaStream_t)stream);
        if (err != cudaSuccess) return WQ_ERR_CUDA;
    }
    return WQ_OK;
}

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

wq_status wq_norm_rope(int n, int n_heads, int head_dim, const wq_head_norm *norm,
                       const wq_rope_axes *rope, const float *x, int64_t x_stride, int out_type,
                       void *out, int64_t out_stride, wq_stream_t stream) {
    NormView nv;
    AxesView ax;
    if (n <= 0 || n_heads <= 0 || !norm_ok(norm, nv) || !axes_ok(rope, head_dim, ax))
        return WQ_ERR_INVALID_ARG;
    if (!float_type(out_type) || !rows_ok(x, x_stride, n_heads, head_dim) ||
        !typed_rows_ok(out, out_type, out_stride, n_heads, head_dim))
        return WQ_ERR_INVALID_ARG;
    if (out == x && (out_stride != x_stride || out_type != WQ_F32)) return WQ_ERR_INVALID_ARG;
    DeviceInfo dev;
    if (!device_info(dev)) return WQ_ERR_CUDA;
    ax.status = dev.status;
    return cuda_status(launch_norm_rope(ax, nv, n, n_heads, head_dim, x, x_stride, out_type, out,
                                        out_stride, dev, (cudaStream_t)stream));
}

size_t wq_norm_rope_grad_workspace_bytes(int n, int n_heads, int head_dim) {
    if (n <= 0 || n_heads <= 0 || head_dim <= 0 || head_dim > kMaxHeadDim) return 0;
    return (size_t)kGradBlocks * 2 * head_dim * sizeof(float);
}

wq_status wq_norm_rope_grad(int n, int n_heads, int head_dim, const wq_head_norm *norm,
                            const wq_rope_axes *rope, const float *x, int64_t x_stride,
                            const float *grad_out, int64_t grad_out_stride, float *grad_x,
                            int64_t grad_x_stride, float *grad_weight, float *grad_bias,
                            void *workspace, size_t workspace_bytes, wq_stream_t stream) {
    NormView nv;
    AxesView ax;
    if (n <= 0 || n_heads <= 0 || !norm_ok(norm, nv) || !axes_ok(rope, head_dim, ax))
        return WQ_ERR_INVALID_ARG;
    if (!rows_ok(x, x_stride, n_heads, head_dim) ||
        !rows_ok(grad_out, grad_out_stride, n_heads, head_dim) ||
        !rows_ok(grad_x, grad_x_stride, n_heads, head_dim))
        return WQ_ERR_INVALID_ARG;
    if ((grad_x == x && grad_x_stride != x_stride) ||
        (grad_x == grad_out && grad_x_stride != grad_out_stride))
        return WQ_ERR_INVALID_ARG;
    const bool sums = grad_weight || grad_bias;
    if (sums && nv.kind == WQ_HEAD_NONE) return WQ_ERR_INVALID_ARG;
    if (!aligned(grad_weight, 4) || !aligned(grad_bias, 4)) return WQ_ERR_INVALID_ARG;
    if (!workspace_ok(workspace, workspace_bytes,
                      sums ? wq_norm_rope_grad_workspace_bytes(n, n_heads, head_dim) : 0))
        return WQ_ERR_INVALID_ARG;
    if ((long long)n * n_heads > 0x7FFFFFFF) return WQ_ERR_TOO_LARGE;
    DeviceInfo dev;
    if (!device_info(dev)) return WQ_ERR_CUDA;
    ax.status = dev.status;
    return cuda_status(launch_norm_rope_grad(ax, nv, n, n_heads, head_dim, x, x_stride, grad_out,
                                             grad_out_stride, grad_x, grad_x_stride, grad_weight,
                                             grad_bias, workspace, dev, (cudaStream_t)stream));
}

wq_status wq_kv_append_norm(const wq_kv_cache *cache, int n_tok, int h_q,
                            const wq_head_norm *q_norm, const wq_head_norm *k_norm,
                            const wq_rope_axes *rope, const float *q, int64_t q_stride,
                            const float *k, int64_t k_stride, const float *v, int64_t v_stride,
                            int n_seq, const int32_t *seq, const int32_t *slot,
                            const int32_t *page_table, int max_pages, int q_type, void *q_out,
                            int64_t q_out_stride, float *acc, int32_t *slot_pos,
                            int64_t acc_stride, wq_stream_t stream) {
    KvView kv;
    NormView qn, kn;
    AxesView ax;
    if (!view_of(cache, n_seq, page_table, max_pages, kv)) return WQ_ERR_INVALID_ARG;
    if (n_tok <= 0 || h_q < 0 || !page_table || !slot || (!seq && n_seq < n_tok))
        return WQ_ERR_INVALID_ARG;
    if (!norm_ok(q_norm, qn) || !norm_ok(k_norm, kn) || !axes_ok(rope, kv.head_dim, ax))
        return WQ_ERR_INVALID_ARG;
    if (!rows_ok(k, k_stride, kv.n_heads, kv.head_dim) ||
        !rows_ok(v, v_stride, kv.n_heads, kv.head_dim))
        return WQ_ERR_INVALID_ARG;
    if (h_q > 0 && (!float_type(q_type) || !rows_ok(q, q_stride, h_q, kv.head_dim) ||
                    !typed_rows_ok(q_out, q_type, q_out_stride, h_q, kv.head_dim) ||
                    (q_out == q && (q_out_stride != q_stride || q_type != WQ_F32))))
        return WQ_ERR_INVALID_ARG;
    if ((acc || slot_pos) && acc_stride < 1) return WQ_ERR_INVALID_ARG;
    if (slot_pos && ax.rot == 0) return WQ_ERR_INVALID_ARG;
    DeviceInfo dev;
    if (!device_info(dev)) return WQ_ERR_CUDA;
    ax.status = dev.status;
    AppendNormArgs a{};
    a.n_tok = n_tok;
    a.h_q = h_q;
    a.n_seq = n_seq;
    a.n_slots = max_pages * (int)kv.page_size.d;
    if (acc || slot_pos) a.n_slots = cut(a.n_slots, acc_stride);
    a.q_type = h_q > 0 ? q_type : WQ_F32;
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
    return cuda_status(launch_append_norm(ax, qn, kn, a, kv, dev, (cudaStream_t)stream));
}

size_t wq_attn_tokens_workspace_bytes(const wq_kv_cache *cache, int n_seq, int n_tok, int h_q,
                                      int q_type) {
    KvView kv;
    if (!view_of(cache, n_seq, nullptr, 1, kv) || n_tok <= 0 || h_q <= 0 || h_q % kv.n_heads ||
        !float_type(q_type) || (long long)n_tok * h_q > kMaxSlots)
        return 0;
    return tokens_workspace_bytes(kv, n_seq, n_tok, h_q, q_type);
}

wq_status wq_attn_tokens(const wq_kv_cache *cache, int n_seq, int n_tok, int h_q, float scale,
                         const wq_attn_form *form, int q_type, const void *q, int64_t q_stride,
                         const int32_t *starts, const int32_t *page_table, int max_pages,
                         const int32_t *lens, int out_type, void *out, int64_t out_stride,
                         float *lse, void *workspace, size_t workspace_bytes,
                         wq_stream_t stream) {
    KvView kv;
    if (!view_of(cache, n_seq, page_table, max_pages, kv)) return WQ_ERR_INVALID_ARG;
    if (n_tok <= 0 || h_q <= 0 || h_q % kv.n_heads || !std::isfinite(scale) ||
        (long long)n_tok * h_q > kMaxSlots)
        return WQ_ERR_INVALID_ARG;
    if (!float_type(q_type) || (out_type != q_type && out_type != WQ_F32))
        return WQ_ERR_INVALID_ARG;
    if (!starts || !page_table || !lens) return WQ_ERR_INVALID_ARG;
    if (!typed_rows_ok(q, q_type, q_stride, h_q, kv.head_dim) ||
        !typed_rows_ok(out, out_type, out_stride, h_q, kv.head_dim))
        return WQ_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(out, 16) || q_stride * element_bytes(q_type) % 16 ||
        out_stride * element_bytes(out_type) % 16)
        return WQ_ERR_INVALID_ARG;
    wq_attn_form f{};
    if (form) f = *form;
    if (!std::isfinite(f.softcap) || f.softcap < 0.f || f.window < 0) return WQ_ERR_INVALID_ARG;
    if (std::fabs(scale) > kMostScale || f.softcap > kMostScale ||
        (f.softcap > 0.f && f.softcap < 1.f / kMostScale))
        return WQ_ERR_INVALID_ARG;
    if ((f.tree && (f.prefix || f.tree_stride < 1 || f.tree_stride > kMaxStride)) ||
        (f.pos && !f.tree))
        return WQ_ERR_INVALID_ARG;
    if (!workspace_ok(workspace, workspace_bytes,
                      tokens_workspace_bytes(kv, n_seq, n_tok, h_q, q_type)))
        return WQ_ERR_INVALID_ARG;
    DeviceInfo dev;
    if (!device_info(dev)) return WQ_ERR_CUDA;
    TokensArgs a{};
    a.n_seq = n_seq;
    a.n_tok = n_tok;
    a.h_q = h_q;
    a.n_slots = max_pages * (int)kv.page_size.d;
    a.group = make_fast_div((uint32_t)(h_q / kv.n_heads));
    a.scale = scale;
    a.softcap = f.softcap;
    a.window = f.window;
    a.slopes = f.slopes;
    a.first = f.first;
    a.prefix = f.prefix;
    a.pos = f.pos;
    a.tree = f.tree;
    a.tree_stride = f.tree_stride;
    a.q_type = q_type;
    a.out_type = out_type;
    a.wide_out = aligned(out, 32) && out_stride * element_bytes(out_type) % 32 == 0 &&
                 kv.head_dim * element_bytes(out_type) % 32 == 0;
    a.q = q;
    a.out = out;
    a.q_stride = q_stride;
    a.out_stride = out_stride;
    a.starts = starts;
    a.lens = lens;
    a.lse = lse;
    a.workspace = workspace;
    a.status = dev.status;
    a.wait_limit = wait_limit();
    return cuda_status(launch_attn_tokens(a, kv, dev, (cudaStream_t)stream));
}

wq_status wq_kv_accept(const wq_kv_cache *caches, int n_caches, int n_seq, int n_tok,
                       const int32_t *page_table, int max_pages, const int32_t *starts,
                       const int32_t *parent, const int32_t *tokens, const int32_t *choice,
                       const int32_t *lens, int32_t *path, int32_t *accepted, int32_t *next,
                       int32_t *lens_out, wq_stream_t stream) {
    return accept_paths(caches, n_caches, n_seq, n_tok, page_table, max_pages, starts, parent,
                        tokens, choice, lens, path, accepted, next, lens_out, nullptr, 0, stream);
}

wq_status wq_kv_accept_slots(const wq_kv_cache *caches, int n_caches, int n_seq, int n_tok,
                             const int32_t *page_table, int max_pages, const int32_t *starts,
                             const int32_t *parent, const int32_t *tokens, const int32_t *choice,
                             const int32_t *lens, int32_t *path, int32_t *accepted, int32_t *next,
                             int32_t *lens_out, const wq_slot_arrays *slots, int64_t acc_stride,
                             wq_stream_t stream) {
    if (!slots || acc_stride < 1) return WQ_ERR_INVALID_ARG;
    return accept_paths(caches, n_caches, n_seq, n_tok, page_table, max_pages, starts, parent,
                        tokens, choice, lens, path, accepted, next, lens_out, slots, acc_stride,
                        stream);
}

}  // extern "C"
