// Shared pieces of the state space scan kernels (gdn_ssm_*.cu): the cut of the
// sequences into segments, the step size and decay of a token, bf16 splitting.
#pragma once

#include "gdn_common.cuh"
#include "gdn_internal.h"

namespace gdn {
namespace ssm {

// The sequences are cut into segments of `seg_len` tokens (at least one per
// sequence, also where it is empty), numbered through all sequences.  Without
// cu_seqlens the map is arithmetic; with it plan_kernel writes the table.
struct SegMap {
    const int4 *table;      // [bound] {sequence, first token, tokens, index in sequence}, or null
    const int *first;       // [N + 1] first segment of each sequence (with the table)
    int N, nseg;            // sequences; segments per sequence (without the table)
    int64_t T;              // tokens per sequence (without the table)
    int seg_len;
    const int *order;       // [bound] which segment a CTA takes, the longest first, or null: in their order
};
// A table of more segments than this stays in its order: the work then evens out by itself.
constexpr int kOrdered = 1024;

struct Seg {
    int n, idx, len;        // sequence, index in it, tokens
    int64_t t0;             // first token (row of the packed batch)
    bool ok, last;
};

// segment of the s-th CTA (of each head's); s becomes the segment's number
__device__ __forceinline__ Seg find_seg(const SegMap &m, int &s) {
    Seg r;
    if (m.table) {
        if (m.order) s = m.order[s];
        r.ok = s < m.first[m.N];
        if (!r.ok) return r;
        const int4 e = m.table[s];
        r.n = e.x;
        r.t0 = e.y;
        r.len = e.z;
        r.idx = e.w;
        r.last = s + 1 == m.first[r.n + 1];
    } else {
        r.ok = true;
        r.n = s / m.nseg;
        r.idx = s - r.n * m.nseg;
        const int64_t at = (int64_t)r.idx * m.seg_len;
        const int64_t left = m.T - at;
        r.len = (int)(left < m.seg_len ? left : m.seg_len);
        r.t0 = (int64_t)r.n * m.T + at;
        r.last = r.idx + 1 == m.nseg;
    }
    return r;
}

// Segment table of a packed batch; the chaining of the segments (gdn_ssm_rows.cu).
cudaError_t launch_plan(const int32_t *cu, int N, int seg_len, int bound, int4 *table, int *first, int *order,
                        cudaStream_t stream);
cudaError_t launch_combine(float *seg_state, const float *seg_decay, const float *h0, float *hT, int N, int HV, int elems,
                           bool whole, const SegMap &map, cudaStream_t stream);
// the tensor-core scan (gdn_ssm_tc.cu)
bool tc_supported(const SsmArgs &a);
size_t tc_workspace_bytes(const SsmArgs &a);
cudaError_t launch_tc(const SsmArgs &a, cudaStream_t stream);

// Dependent launches: a kernel launched with launch_after may start while the one
// before it in the stream still runs; wait_for_previous() returns when that one is done
// (and with it all before it), let_next_start() lets the next one start early.
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
template <typename... P, typename... A>
cudaError_t launch_after(void (*kern)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream, A &&...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t err = cudaLaunchKernelEx(&cfg, kern, static_cast<P>(args)...);
    return err == cudaSuccess ? cudaGetLastError() : err;
}

// log(1 + e^x), finite and accurate at both ends
__device__ __forceinline__ float softplus(float x) { return fmaxf(x, 0.f) + log1pf(expf(-fabsf(x))); }

// step size of one token and head
__device__ __forceinline__ float step_size(float dt, float bias, bool soft) {
    const float v = dt + bias;
    return soft ? softplus(v) : v;
}

}  // namespace ssm
}  // namespace gdn
