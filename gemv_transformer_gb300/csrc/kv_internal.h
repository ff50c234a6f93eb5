// kv_internal.h -- host-side declarations of the rotary and paged-cache calls.
#pragma once

#include "kv_cache.cuh"
#include "wq_internal.h"

namespace wq {

struct RopeArgs {
    int head_dim, rot;
    unsigned flags;
    const int32_t *pos;   // [n]; may be null when rot == 0
    const float2 *table;  // [table_rows][rot/2]
    int table_rows;
    unsigned *status;
};

struct AppendArgs {
    RopeArgs rope;
    int n_tok, h_q, n_seq;
    int n_slots;  // max_pages * page_size, cut to acc_stride when there are sums
    const float *q, *k, *v;
    long long q_stride, k_stride, v_stride, q_out_stride;
    float *q_out;
    const int32_t *seq, *slot;
    float *acc;
    int32_t *slot_pos;
    long long acc_stride;
};

struct AttnArgs {
    int n_seq, h_q, group;  // group: query heads per kv head
    int n_slots;            // max_pages * page_size, cut to the given strides
    float scale;
    int window;
    const float *q;
    const int32_t *lens;
    const float *mask;
    float *out, *lse;
    const float *acc_in;
    float *acc_out;
    long long q_stride, mask_stride, out_stride, acc_stride;
    void *workspace;
    unsigned *status;
};

struct EvictArgs {
    int n_seq, n_slots, keep, sinks, recent;
    const int32_t *lens, *seen;
    const float *acc;
    const int32_t *slot_pos;
    float *acc_out;
    int32_t *pos_out, *lens_out;
    long long acc_stride;
    void *workspace;
    unsigned *status;
};

cudaError_t launch_rope_table(int rows, int rot, double base, const wq_rope_scaling &sc,
                              float *table, const DeviceInfo &dev, cudaStream_t stream);
cudaError_t launch_rope(const RopeArgs &r, const float *x, long long x_stride, int n, int n_heads,
                        float *out, long long out_stride, const DeviceInfo &dev,
                        cudaStream_t stream);
cudaError_t launch_kv_append(const AppendArgs &a, const KvView &kv, const DeviceInfo &dev,
                             cudaStream_t stream);
size_t attn_workspace_bytes(const KvView &kv, int n_seq, int h_q, int n_slots, bool with_acc);
cudaError_t launch_attn_paged(const AttnArgs &a, const KvView &kv, const DeviceInfo &dev,
                              cudaStream_t stream);
size_t evict_workspace_bytes(const KvView &kv, int n_seq, int n_slots, int keep);
cudaError_t launch_kv_evict(const EvictArgs &a, const KvView &kv, const DeviceInfo &dev,
                            cudaStream_t stream);

}  // namespace wq
