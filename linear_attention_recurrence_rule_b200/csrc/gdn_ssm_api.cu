// C ABI entry points of the state space scan, its single-token step and the norms
// around a block (declared in include/gdn.h): argument validation and dispatch.
#include <cuda_runtime.h>

#include <cmath>

#include "gdn.h"
#include "gdn_internal.h"

namespace {

bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool known(gdn_dtype d) { return d == GDN_F32 || d == GDN_BF16; }
int elt(gdn_dtype d) { return d == GDN_BF16 ? 2 : 4; }
constexpr int64_t kGrid = 0x7fffffff;

// sizes only (shared with the workspace query)
gdn_status check_ssm_sizes(int N, int64_t T, int HK, int HV, int dk, int dv, gdn_dtype dtype) {
    if (N < 0 || T < 0 || HK <= 0 || HV <= 0 || dk <= 0 || dv <= 0 || HV % HK) return GDN_ERR_INVALID_ARG;
    if (!known(dtype)) return GDN_ERR_INVALID_ARG;
    if (!gdn::ssm_supported(dk, dv)) return GDN_ERR_UNSUPPORTED;
    if ((int64_t)HV * dv > kGrid || (int64_t)HK * dk > kGrid) return GDN_ERR_UNSUPPORTED;
    // grid.x: up to 4 CTAs for each segment's state; cutting adds some hundred states at most
    if ((int64_t)N * HV > kGrid / 8) return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}

gdn_status check_step_sizes(int N, int HK, int HV, int dk, int dv) {
    if (N < 0 || HK <= 0 || HV <= 0 || dk <= 0 || dv <= 0 || HV % HK) return GDN_ERR_INVALID_ARG;
    if (!gdn::decode_supported(dk, dv)) return GDN_ERR_UNSUPPORTED;
    // the row, rounded up to a block of 256 channels, in 32 bits; sequences in groups of four
    // over grid.y
    if ((int64_t)N * HV > kGrid || (int64_t)HV * dv + 2 * (int64_t)HK * dk > kGrid - 255 || N > 4 * 65535)
        return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}

}  // namespace

extern "C" {

size_t gdn_ssm_step_workspace_size(int N, int HK, int HV, int dk, int dv) {
    return check_step_sizes(N, HK, HV, dk, dv) == GDN_OK ? gdn::ssm_step_workspace_bytes(N, HK, HV, dk, dv) : 0;
}

size_t gdn_ssm_prefill_workspace_size(int N, int64_t T, int HK, int HV, int dk, int dv, gdn_dtype dtype,
                                      int varlen) {
    if (check_ssm_sizes(N, T, HK, HV, dk, dv, dtype) != GDN_OK || N == 0) return 0;
    gdn::SsmArgs a{};
    a.N = N;
    a.T = T;
    a.HK = HK;
    a.HV = HV;
    a.dk = dk;
    a.dv = dv;
    a.dtype = dtype;
    static const int32_t some = 0;
    a.cu_seqlens = varlen ? &some : nullptr;
    return gdn::ssm_workspace_bytes(a);
}

gdn_status gdn_ssm_prefill(const void *x, const void *b, const void *c, const float *dt, const float *a,
                           const float *d, const float *dt_bias, const float *h0,
                           const int32_t *cu_seqlens, int N, int64_t T, int HK, int HV, int dk, int dv,
                           int64_t x_row, int64_t b_row, int64_t c_row, unsigned flags, gdn_dtype dtype,
                           void *y, float *hT, void *workspace, size_t workspace_bytes,
                           gdn_stream_t stream) {
    if (flags & ~GDN_SSM_SOFTPLUS) return GDN_ERR_INVALID_ARG;
    const gdn_status st = check_ssm_sizes(N, T, HK, HV, dk, dv, dtype);
    if (st != GDN_OK) return st;
    if (N == 0) return GDN_OK;   // empty batch: buffers may be NULL
    if (!a || (T > 0 && (!x || !b || !c || !dt || !y))) return GDN_ERR_INVALID_ARG;
    if (x_row == 0) x_row = (int64_t)HV * dv;
    if (b_row == 0) b_row = (int64_t)HK * dk;
    if (c_row == 0) c_row = (int64_t)HK * dk;
    if (x_row < (int64_t)HV * dv || b_row < (int64_t)HK * dk || c_row < (int64_t)HK * dk)
        return GDN_ERR_INVALID_ARG;
    const int64_t tokens = cu_seqlens ? T : T > 0 && N > ((int64_t)1 << 40) / T ? -1 : (int64_t)N * T;
    if (tokens < 0 || tokens > kGrid) return GDN_ERR_UNSUPPORTED;
    const int e = elt(dtype);
    if (!aligned(x, 16) || !aligned(b, 16) || !aligned(c, 16) || !aligned(y, 16) || !aligned(h0, 16) ||
        !aligned(hT, 16) || x_row * e % 16 || b_row * e % 16 || c_row * e % 16)
        return GDN_ERR_ALIGNMENT;
    if (!aligned(dt, 4) || !aligned(a, 4) || !aligned(d, 4) || !aligned(dt_bias, 4) || !aligned(cu_seqlens, 4))
        return GDN_ERR_ALIGNMENT;
    gdn::SsmArgs s{x, b, c, dt, a, d, dt_bias, h0, cu_seqlens, N, T, HK, HV, dk, dv, x_row, b_row, c_row,
                   dtype, (flags & GDN_SSM_SOFTPLUS) != 0, y, hT, workspace, workspace_bytes};
    const size_t need = gdn::ssm_workspace_bytes(s);
    if (need > 0 && (!workspace || workspace_bytes < need)) {
        if (gdn::ssm_uses_workspace(s)) return GDN_ERR_WORKSPACE;
        s.workspace = nullptr;   // room for smaller calls only; this one leaves no status either
    }
    if (!aligned(workspace, 16)) return GDN_ERR_ALIGNMENT;
    const cudaError_t err = gdn::launch_ssm_prefill(s, reinterpret_cast<cudaStream_t>(stream));
    return err == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

gdn_status gdn_ssm_step(const void *xbc, const float *dt, const float *a, const float *d,
                        const float *dt_bias, const float *conv_weight, const float *conv_bias,
                        const void *conv_state, void *conv_state_out, int conv_width,
                        const float *state, float *state_out, int N, int HK, int HV, int dk, int dv,
                        int64_t xbc_row, unsigned flags, gdn_dtype dtype, void *y, void *workspace,
                        size_t workspace_bytes, gdn_stream_t stream) {
    if (flags & ~(GDN_SSM_SOFTPLUS | GDN_CONV_SILU)) return GDN_ERR_INVALID_ARG;
    const gdn_status st = check_step_sizes(N, HK, HV, dk, dv);
    if (st != GDN_OK) return st;
    if (!known(dtype)) return GDN_ERR_INVALID_ARG;
    const int64_t C = (int64_t)HV * dv + 2 * (int64_t)HK * dk;
    if (conv_weight && (conv_width < 2 || conv_width > GDN_CONV_MAX_WIDTH)) return GDN_ERR_UNSUPPORTED;
    if (N == 0) return GDN_OK;   // empty batch: buffers may be NULL
    if (!xbc || !dt || !a || !state || !state_out || !y) return GDN_ERR_INVALID_ARG;
    if (conv_weight && (!conv_state || !conv_state_out)) return GDN_ERR_INVALID_ARG;
    if (xbc_row == 0) xbc_row = C;
    if (xbc_row < C) return GDN_ERR_INVALID_ARG;
    if (!aligned(state, 16) || !aligned(state_out, 16)) return GDN_ERR_ALIGNMENT;
    const int e = elt(dtype);
    if (!aligned(xbc, e) || !aligned(y, e) || !aligned(conv_state, e) || !aligned(conv_state_out, e) ||
        !aligned(dt, 4) || !aligned(a, 4) || !aligned(d, 4) || !aligned(dt_bias, 4) ||
        !aligned(conv_weight, 4) || !aligned(conv_bias, 4))
        return GDN_ERR_ALIGNMENT;
    if (!workspace || workspace_bytes < gdn::ssm_step_workspace_bytes(N, HK, HV, dk, dv)) return GDN_ERR_WORKSPACE;
    if (!aligned(workspace, 16)) return GDN_ERR_ALIGNMENT;
    gdn::SsmStepArgs s{xbc, dt, a, d, dt_bias, conv_weight, conv_bias, conv_state, conv_state_out,
                       conv_width, (flags & GDN_CONV_SILU) != 0, (flags & GDN_SSM_SOFTPLUS) != 0, state,
                       state_out, N, HK, HV, dk, dv, xbc_row, dtype, y, workspace};
    const cudaError_t err = gdn::launch_ssm_step(s, reinterpret_cast<cudaStream_t>(stream));
    return err == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

gdn_status gdn_gated_norm(const void *o, const void *z, const float *weight, int64_t rows, int G, int D,
                          int64_t o_row, int64_t z_row, int weight_groups, float eps, unsigned flags,
                          gdn_dtype dtype, void *y, gdn_stream_t stream) {
    if (flags & ~(GDN_GATE_SILU | GDN_NORM_GATE_FIRST | GDN_NORM_UNIT_OFFSET)) return GDN_ERR_INVALID_ARG;
    if (rows < 0 || G <= 0 || D <= 0 || !known(dtype)) return GDN_ERR_INVALID_ARG;
    if (weight && weight_groups != 1 && weight_groups != G) return GDN_ERR_INVALID_ARG;
    if (!(eps >= 0.f) || std::isinf(eps)) return GDN_ERR_INVALID_ARG;
    if (D > gdn::kNormMaxWidth || (int64_t)G * D > kGrid || rows > kGrid / G) return GDN_ERR_UNSUPPORTED;
    if (rows == 0) return GDN_OK;   // nothing to do: buffers may be NULL
    if (!o || !y) return GDN_ERR_INVALID_ARG;
    if (o_row == 0) o_row = (int64_t)G * D;
    if (z_row == 0) z_row = (int64_t)G * D;
    if (o_row < (int64_t)G * D || z_row < (int64_t)G * D) return GDN_ERR_INVALID_ARG;
    const int e = elt(dtype);
    if (!aligned(o, e) || !aligned(z, e) || !aligned(y, e) || !aligned(weight, 4)) return GDN_ERR_ALIGNMENT;
    gdn::GatedNormArgs n{o, z, weight, rows, o_row, z_row, G, D, weight && weight_groups == G && G > 1,
                         (flags & GDN_GATE_SILU) != 0, (flags & GDN_NORM_GATE_FIRST) != 0,
                         (flags & GDN_NORM_UNIT_OFFSET) != 0, eps, dtype, y};
    const cudaError_t err = gdn::launch_gated_norm(n, reinterpret_cast<cudaStream_t>(stream));
    return err == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

gdn_status gdn_residual_norm(const void *x, const void *residual, const float *weight,
                             const float *post_weight, const void *z, int64_t rows, int C, float scale,
                             float eps, unsigned flags, gdn_dtype dtype, gdn_dtype residual_dtype,
                             void *residual_out, void *y, gdn_stream_t stream) {
    if (flags & ~(GDN_GATE_SILU | GDN_NORM_UNIT_OFFSET)) return GDN_ERR_INVALID_ARG;
    if (rows < 0 || C <= 0 || !known(dtype) || !known(residual_dtype)) return GDN_ERR_INVALID_ARG;
    if (!(eps >= 0.f) || std::isinf(eps)) return GDN_ERR_INVALID_ARG;
    if (residual_dtype != GDN_F32 && residual_dtype != dtype) return GDN_ERR_UNSUPPORTED;
    if (C > gdn::kNormMaxWidth || rows > kGrid) return GDN_ERR_UNSUPPORTED;
    if (rows == 0) return GDN_OK;   // nothing to do: buffers may be NULL
    if (!x || (!y && !residual_out)) return GDN_ERR_INVALID_ARG;
    const int e = elt(dtype), er = elt(residual_dtype);
    if (!aligned(x, e) || !aligned(z, e) || !aligned(y, e) || !aligned(residual, er) ||
        !aligned(residual_out, er) || !aligned(weight, 4) || !aligned(post_weight, 4))
        return GDN_ERR_ALIGNMENT;
    gdn::ResidualNormArgs n{x, z, residual, post_weight, weight, rows, C, (flags & GDN_GATE_SILU) != 0,
                            (flags & GDN_NORM_UNIT_OFFSET) != 0, scale, eps, dtype, residual_dtype,
                            residual_out, y};
    const cudaError_t err = gdn::launch_residual_norm(n, reinterpret_cast<cudaStream_t>(stream));
    return err == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // extern "C"
