// One token of the selective state space rule for N sequences, with the short
// causal convolution over the token's packed row x | b | c in front of it.
//
//   u_t[ch] = act(bias[ch] + sum_{j<W} w[ch][j] in_{t-(W-1)+j}[ch])     (x | b | c)
//   S <- alpha S + delta x b^T,   y = S c + d x       (delta, alpha as in gdn_ssm_rows.cu)
//
// Two kernels:
//  * step_row_kernel: a thread per channel (four sequences each, its taps loaded
//    once) convolves the row into the workspace in fp32 and moves the carried inputs
//    on -- nobody else reads a channel's inputs, so in place is as good as not; it
//    also forms delta and alpha of every head.
//  * ssm_step_kernel: bound by the states' pass through memory.  Each fp32 element is
//    loaded once (128-bit, streaming) and stored once; a row lies in DK/4 lanes, and a
//    lane issues its NB row loads before anything else.  It is launched as a dependent
//    of the first kernel and loads states while that one still runs: the states do not
//    depend on it.  The rows' sums are reduced transposed (9 shuffles for 8 rows).
#include "gdn_ssm_common.cuh"

namespace gdn {
namespace {

using ssm::let_next_start;
using ssm::step_size;
using ssm::wait_for_previous;

constexpr int kWarps = 8;
constexpr int kRowSeqs = 4;      // sequences per thread of step_row_kernel

struct RowCall {
    const float *dt, *a, *dt_bias, *cw, *cb;
    float *row;              // [N][C]
    float2 *gates;           // [N][HV] delta, alpha
    int64_t xbc_row;
    int N, C, HV;
    bool silu, soft;
};

// W 0: no convolution.  grid.x: blocks of 256 channels, then the heads' gates
template <typename T, int W>
__global__ void __launch_bounds__(256)
step_row_kernel(const T *__restrict__ xbc, const T *cs, T *cs_out, const RowCall p) {
    let_next_start();
    const int cblocks = (p.C + 255) / 256;
    const int n0 = blockIdx.y * kRowSeqs;
    if ((int)blockIdx.x >= cblocks) {
        const int h = ((int)blockIdx.x - cblocks) * 256 + threadIdx.x;
        if (h >= p.HV) return;
        const float ah = p.a[h], bias = p.dt_bias ? p.dt_bias[h] : 0.f;
        for (int n = n0; n < min(n0 + kRowSeqs, p.N); ++n) {
            const float dl = step_size(p.dt[(size_t)n * p.HV + h], bias, p.soft);
            p.gates[(size_t)n * p.HV + h] = make_float2(dl, expf(dl * ah));
        }
        return;
    }
    const int ch = blockIdx.x * 256 + threadIdx.x;
    if (ch >= p.C) return;
    constexpr int H = W > 1 ? W - 1 : 1;
    T hist[kRowSeqs][H], in[kRowSeqs];
    float wt[W > 0 ? W : 1];
#pragma unroll
    for (int i = 0; i < kRowSeqs; ++i) {
        const int n = n0 + i;
        if (n < p.N) {
            in[i] = xbc[(int64_t)n * p.xbc_row + ch];
            if (W > 0)
#pragma unroll
                for (int m = 0; m < W - 1; ++m) hist[i][m] = cs[((size_t)n * (W - 1) + m) * p.C + ch];
        }
    }
    if (W > 0)
#pragma unroll
        for (int m = 0; m < W; ++m) wt[m] = p.cw[(size_t)ch * W + m];
    const float bias = W > 0 && p.cb ? p.cb[ch] : 0.f;
#pragma unroll
    for (int i = 0; i < kRowSeqs; ++i) {
        const int n = n0 + i;
        if (n >= p.N) break;
        float v = to_f32(in[i]);
        if (W > 0) {
            float acc = bias;
#pragma unroll
            for (int m = 0; m < W - 1; ++m) acc = fmaf(wt[m], to_f32(hist[i][m]), acc);
            acc = fmaf(wt[W > 0 ? W - 1 : 0], v, acc);
#pragma unroll
            for (int m = 0; m < W - 1; ++m)
                cs_out[((size_t)n * (W - 1) + m) * p.C + ch] = m + 1 < W - 1 ? hist[i][m + 1 < H ? m + 1 : 0] : in[i];
            // full-precision sigmoid: the convolved value goes into the fp32 state
            v = p.silu ? acc / (1.f + expf(-acc)) : acc;
        }
        p.row[(size_t)n * p.C + ch] = v;
    }
}

// v[8] summed over the lanes of a row (LPR lanes): halves the values three times, then
// plain butterflies; the lane with (its bits LPR/2, LPR/4, LPR/8) = j has row j's sum
template <int LPR>
__device__ __forceinline__ float reduce8(const float (&v)[8], int lane, int &j) {
    float a[4], b[2];
    const bool u0 = lane & (LPR / 2), u1 = lane & (LPR / 4), u2 = lane & (LPR / 8);
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = (u0 ? v[4 + i] : v[i]) + __shfl_xor_sync(0xffffffffu, u0 ? v[i] : v[4 + i], LPR / 2);
#pragma unroll
    for (int i = 0; i < 2; ++i) b[i] = (u1 ? a[2 + i] : a[i]) + __shfl_xor_sync(0xffffffffu, u1 ? a[i] : a[2 + i], LPR / 4);
    float c = (u2 ? b[1] : b[0]) + __shfl_xor_sync(0xffffffffu, u2 ? b[0] : b[1], LPR / 8);
#pragma unroll
    for (int o = LPR / 16; o > 0; o >>= 1) c += __shfl_xor_sync(0xffffffffu, c, o);
    j = (u0 ? 4 : 0) + (u1 ? 2 : 0) + (u2 ? 1 : 0);
    return c;
}

struct StepCall {
    const float *row;
    const float2 *gates;
    const float *d, *state;
    float *state_out;
    int HK, HV, dv;
    size_t C;
};

template <int DK, typename T>
__global__ void __launch_bounds__(kWarps * 32, 4)
ssm_step_kernel(const StepCall p, T *__restrict__ y) {
    constexpr int NB = 8;
    constexpr int LPR = DK / 4;             // lanes per state row
    constexpr int RPI = 32 / LPR;           // rows per warp instruction
    const int nh = blockIdx.x;
    const int n = nh / p.HV, h = nh - n * p.HV, g = h / (p.HV / p.HK);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int col = (lane % LPR) * 4;
    // this warp's NB x RPI consecutive rows
    const int row0 = (blockIdx.y * kWarps + warp) * NB * RPI + lane / LPR * NB;
    const size_t off = (size_t)nh * p.dv * DK + col;
    const float *S = p.state + off;
    float *So = p.state_out + off;
    float4 s[NB];
#pragma unroll
    for (int j = 0; j < NB; ++j)
        s[j] = row0 + j < p.dv ? __ldcs(reinterpret_cast<const float4 *>(S + (size_t)(row0 + j) * DK))
                               : make_float4(0.f, 0.f, 0.f, 0.f);
    wait_for_previous();
    const float *r = p.row + (size_t)n * p.C;
    const float *bc = r + (size_t)p.HV * p.dv + (size_t)g * DK + col;
    // (rows of the packed x | b | c may start anywhere: single loads)
    float b[4], c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        b[i] = __ldcg(bc + i);
        c[i] = __ldcg(bc + (size_t)p.HK * DK + i);
    }
    const float2 gate = __ldcg(p.gates + nh);
    const float dh = p.d ? p.d[h] : 0.f;
    float x[NB], v[NB];
#pragma unroll
    for (int j = 0; j < NB; ++j) x[j] = row0 + j < p.dv ? __ldcg(r + (size_t)h * p.dv + row0 + j) : 0.f;
#pragma unroll
    for (int j = 0; j < NB; ++j) {
        const float u = gate.x * x[j];
        float4 ns;
        ns.x = fmaf(gate.y, s[j].x, u * b[0]);
        ns.y = fmaf(gate.y, s[j].y, u * b[1]);
        ns.z = fmaf(gate.y, s[j].z, u * b[2]);
        ns.w = fmaf(gate.y, s[j].w, u * b[3]);
        if (row0 + j < p.dv) __stcs(reinterpret_cast<float4 *>(So + (size_t)(row0 + j) * DK), ns);
        v[j] = ns.x * c[0] + ns.y * c[1] + ns.z * c[2] + ns.w * c[3];
    }
    int j;
    const float sum = reduce8<LPR>(v, lane, j);
    float xj = x[0];
#pragma unroll
    for (int i = 1; i < NB; ++i) xj = j == i ? x[i] : xj;
    if ((lane & (LPR / 8 - 1)) == 0 && row0 + j < p.dv)
        y[(size_t)nh * p.dv + row0 + j] = from_f32<T>(fmaf(dh, xj, sum));
}

template <typename T, int W>
void launch_row(const SsmStepArgs &a, const RowCall &r, cudaStream_t stream) {
    const dim3 grid((unsigned)((r.C + 255) / 256 + (r.HV + 255) / 256), (unsigned)((a.N + kRowSeqs - 1) / kRowSeqs));
    step_row_kernel<T, W><<<grid, 256, 0, stream>>>(static_cast<const T *>(a.xbc), static_cast<const T *>(a.conv_state),
                                                    static_cast<T *>(a.conv_state_out), r);
}

template <int DK, typename T>
cudaError_t launch_dk(const SsmStepArgs &a, cudaStream_t stream) {
    const int C = a.HV * a.dv + 2 * a.HK * DK;
    float2 *gates = static_cast<float2 *>(a.workspace);
    float *row = reinterpret_cast<float *>(gates + (size_t)a.N * a.HV);
    const RowCall r{a.dt, a.a, a.dt_bias, a.conv_w, a.conv_b, row, gates, a.xbc_row, a.N, C, a.HV,
                    a.conv_silu, a.softplus};
    switch (a.conv_w ? a.conv_width : 0) {
        case 0: launch_row<T, 0>(a, r, stream); break;
        case 2: launch_row<T, 2>(a, r, stream); break;
        case 3: launch_row<T, 3>(a, r, stream); break;
        case 4: launch_row<T, 4>(a, r, stream); break;
        case 5: launch_row<T, 5>(a, r, stream); break;
        case 6: launch_row<T, 6>(a, r, stream); break;
        case 7: launch_row<T, 7>(a, r, stream); break;
        default: launch_row<T, 8>(a, r, stream); break;
    }
    cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess) return err;
    constexpr int BAND = kWarps * (32 / (DK / 4)) * 8;
    const dim3 grid((unsigned)(a.N * a.HV), (unsigned)((a.dv + BAND - 1) / BAND));
    const StepCall s{row, gates, a.d, a.state, a.state_out, a.HK, a.HV, a.dv, (size_t)C};
    return ssm::launch_after(ssm_step_kernel<DK, T>, grid, dim3(kWarps * 32), 0, stream, s, static_cast<T *>(a.y));
}

template <typename T>
cudaError_t launch_typed(const SsmStepArgs &a, cudaStream_t stream) {
    switch (a.dk) {
        case 32: return launch_dk<32, T>(a, stream);
        case 64: return launch_dk<64, T>(a, stream);
        default: return launch_dk<128, T>(a, stream);
    }
}

}  // namespace

size_t ssm_step_workspace_bytes(int N, int HK, int HV, int dk, int dv) {
    return (size_t)N * ((size_t)HV * sizeof(float2) + ((size_t)HV * dv + 2 * (size_t)HK * dk) * sizeof(float));
}

cudaError_t launch_ssm_step(const SsmStepArgs &a, cudaStream_t stream) {
    return a.dtype == GDN_BF16 ? launch_typed<__nv_bfloat16>(a, stream) : launch_typed<float>(a, stream);
}

}  // namespace gdn
