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

// A norm of heads as the kernels see it.
struct NormView {
    int kind;  // WQ_HEAD_*
    float eps;
    const float *weight, *bias;
};

// Rotary positions on several axes: pair i by column code[i] & 255 at the position on axis
// code[i] >> 8.
struct AxesView {
    int rot;
    unsigned flags;  // WQ_ROPE_INTERLEAVED
    int axes;        // 0 where rot is 0
    unsigned used;   // bit a: axis a has pairs
    int table_rows, table_pairs;
    bool straight;   // pair i by column i on axis 0, columns in 16-byte runs
    const int32_t *pos;
    long long pos_stride;
    const float2 *table;
    unsigned *status;
    uint16_t code[128];
};

struct AppendNormArgs {
    int n_tok, h_q, n_seq, n_slots, q_type;
    const float *q, *k, *v;
    long long q_stride, k_stride, v_stride, q_out_stride;
    void *q_out;
    const int32_t *seq, *slot;
    float *acc;
    int32_t *slot_pos;
    long long acc_stride;
};

constexpr int kGradBlocks = 608;  // four on each of 152 SMs: all at once

struct TokensArgs {
    int n_seq, n_tok, h_q, n_slots;  // n_slots: max_pages * page_size
    FastDiv group;                   // query heads per kv head
    float scale, softcap;
    int window;
    const float *slopes;
    const int32_t *first, *prefix, *pos;
    const uint32_t *tree;
    long long tree_stride;
    int q_type, out_type;
    bool wide_out;     // rows of out in whole 32-byte runs
    bool join_inside;  // parts of row tiles are joined by the last of their CTAs, not by a launch
    const void *q;
    void *out;
    long long q_stride, out_stride;  // in elements
    const int32_t *starts, *lens;
    float *lse;
    void *workspace;
    unsigned *status;
    unsigned long long wait_limit;
};

struct AcceptArgs {
    int n_seq, n_tok, n_slots;
    const int32_t *starts, *parent, *tokens, *choice, *lens;
    int32_t *path, *accepted, *next, *lens_out;
    unsigned *status;
};
// The pools of up to kAcceptCaches layers; the rest of their description is the first's.
constexpr int kAcceptCaches = 48;
struct AcceptPools {
    int count;
    char *k[kAcceptCaches], *v[kAcceptCaches];
};
// Their slots' weights and positions, by turns, each [n_seq][kv heads][stride] or null.
struct AcceptSlots {
    long long stride, seq0;  // seq0: the launch's first sequence
    void *p[2 * kAcceptCaches];
};

cudaError_t launch_norm_rope(const AxesView &ax, const NormView &nv, int n, int n_heads,
                             int head_dim, const float *x, long long x_stride, int out_type,
                             void *out, long long out_stride, const DeviceInfo &dev,
                             cudaStream_t stream);
cudaError_t launch_append_norm(const AxesView &ax, const NormView &q_norm, const NormView &k_norm,
                               const AppendNormArgs &a, const KvView &kv, const DeviceInfo &dev,
                               cudaStream_t stream);
// workspace: kGradBlocks * 2 * head_dim floats where a sum is wanted.
cudaError_t launch_norm_rope_grad(const AxesView &ax, const NormView &nv, int n, int n_heads,
                                  int head_dim, const float *x, long long x_stride,
                                  const float *grad, long long grad_stride, float *grad_x,
                                  long long grad_x_stride, float *grad_weight, float *grad_bias,
                                  void *workspace, const DeviceInfo &dev, cudaStream_t stream);
size_t tokens_workspace_bytes(const KvView &kv, int n_seq, int n_tok, int h_q, int q_type);
cudaError_t launch_attn_tokens(const TokensArgs &a, const KvView &kv, const DeviceInfo &dev,
                               cudaStream_t stream);
// slots: null where there are none.
cudaError_t launch_kv_accept(const AcceptArgs &a, const KvView &kv, const AcceptPools &pools,
                             const AcceptSlots *slots, bool write_path, cudaStream_t stream);

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
