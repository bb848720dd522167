// One token of the selective state space rule for N sequences, with the short
// causal convolution over the token's packed row x | b | c in front of it.
//
//   u_t[ch] = act(bias[ch] + sum_{j<W} w[ch][j] in_{t-(W-1)+j}[ch])     (x | b | c)
//   S <- alpha S + delta x b^T,   y = S c + d x       (delta, alpha as in gdn_ssm_rows.cu)
//
// Bound by the states' pass through memory: each fp32 element is loaded once
// (128-bit, streaming) and stored once.  CTAs of 8 warps own a band of rows of one
// (sequence, head) state, a row in DK/4 lanes; every lane has NB loads in flight
// before anything else, and the convolution's loads (its 2 DK + band channels, W
// taps) go out behind them, so that they cost no time of their own.  Each CTA of a
// group convolves the group's b and c itself: W taps of 2 DK channels from L2 are
// far less than its 32 KB of state.
//
// The carried inputs of the x channels belong to one CTA and move in place.  Those
// of b and c are read by every CTA of the group: where they move in place, a small
// second kernel does it; otherwise the group's first CTA writes them.
#include "gdn_ssm_common.cuh"

namespace gdn {
namespace {

using ssm::step_size;

constexpr int kWarps = 8;
constexpr int kMaxBand = 128;

template <typename T>
struct StepParams {
    const T *xbc;
    const float *dt, *a, *d, *dt_bias, *cw, *cb;
    const T *cs;
    T *cs_out;
    const float *state;
    float *state_out;
    T *y;
    int HK, HV, dv, W;       // W 0: no convolution
    int64_t row;
    bool conv_silu, soft;
    bool move_bc;            // the carried inputs of b and c are written here (not in place)
};

// the convolution of one channel for the sequence's new token; `move`: its carried
// inputs go on by one token
template <typename T>
__device__ __forceinline__ float conv_channel(const StepParams<T> &p, int n, size_t C, int ch, bool move) {
    const T in = p.xbc[(int64_t)n * p.row + ch];
    const float vin = to_f32(in);
    if (p.W == 0) return vin;
    constexpr int MW = kConvMaxWidth;
    const int W = p.W;
    const T *cs = p.cs + (size_t)n * (W - 1) * C + ch;
    const float *wr = p.cw + (size_t)ch * W;
    T hist[MW - 1];
    float wt[MW];
#pragma unroll
    for (int m = 0; m < MW - 1; ++m)
        if (m < W - 1) hist[m] = cs[m * C];
#pragma unroll
    for (int m = 0; m < MW; ++m)
        if (m < W) wt[m] = wr[m];
    float acc = p.cb ? p.cb[ch] : 0.f;
#pragma unroll
    for (int m = 0; m < MW - 1; ++m)
        if (m < W - 1) acc = fmaf(wt[m], to_f32(hist[m]), acc);
#pragma unroll
    for (int m = 0; m < MW; ++m)
        if (m == W - 1) acc = fmaf(wt[m], vin, acc);
    if (move) {
        T *co = p.cs_out + (size_t)n * (W - 1) * C + ch;
#pragma unroll
        for (int m = 0; m < MW - 2; ++m)
            if (m < W - 2) co[m * C] = hist[m + 1];
        co[(W - 2) * C] = in;
    }
    // full-precision sigmoid: the convolved value goes into the fp32 state
    return p.conv_silu ? acc / (1.f + expf(-acc)) : acc;
}

template <int DK, int NB, typename T>
__global__ void __launch_bounds__(kWarps * 32, NB >= 8 ? 3 : 4)
ssm_step_kernel(const StepParams<T> p) {
    constexpr int LPR = DK / 4;             // lanes per state row
    constexpr int RPI = 32 / LPR;           // rows per warp instruction
    constexpr int BAND = kWarps * RPI * NB;
    __shared__ float sb[DK], sc[DK], sx[BAND];
    const int nh = blockIdx.x;
    const int n = nh / p.HV, h = nh - n * p.HV;
    const int R = p.HV / p.HK, g = h / R;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int sub = lane / LPR, col = (lane % LPR) * 4;
    const int base = blockIdx.y * BAND;
    const size_t off = (size_t)nh * p.dv * DK;
    const float *S = p.state + off;
    float *So = p.state_out + off;

    float4 s[NB];
#pragma unroll
    for (int j = 0; j < NB; ++j) {
        const int row = base + (j * kWarps + warp) * RPI + sub;
        s[j] = row < p.dv ? __ldcs(reinterpret_cast<const float4 *>(S + (size_t)row * DK + col))
                          : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    const float delta = step_size(p.dt[nh], p.dt_bias ? p.dt_bias[h] : 0.f, p.soft);
    const float alpha = expf(delta * p.a[h]);
    const float dh = p.d ? p.d[h] : 0.f;
    const size_t C = (size_t)p.HV * p.dv + 2 * (size_t)p.HK * DK;
    const int rows = min(BAND, p.dv - base);
    const bool move_bc = p.move_bc && h == g * R && blockIdx.y == 0;
    for (int i = threadIdx.x; i < 2 * DK + rows; i += kWarps * 32) {
        if (i < 2 * DK) {
            const bool isc = i >= DK;
            const int ch = p.HV * p.dv + (isc ? p.HK * DK : 0) + g * DK + (isc ? i - DK : i);
            (isc ? sc[i - DK] : sb[i]) = conv_channel(p, n, C, ch, move_bc);
        } else {
            const int r = i - 2 * DK;
            sx[r] = conv_channel(p, n, C, h * p.dv + base + r, p.W > 0);
        }
    }
    __syncthreads();
    const float4 b = *reinterpret_cast<const float4 *>(sb + col);
    const float4 c = *reinterpret_cast<const float4 *>(sc + col);
#pragma unroll
    for (int j = 0; j < NB; ++j) {
        const int r = (j * kWarps + warp) * RPI + sub, row = base + r;
        const float x = row < p.dv ? sx[r] : 0.f;
        const float u = delta * x;
        float4 ns;
        ns.x = fmaf(alpha, s[j].x, u * b.x);
        ns.y = fmaf(alpha, s[j].y, u * b.y);
        ns.z = fmaf(alpha, s[j].z, u * b.z);
        ns.w = fmaf(alpha, s[j].w, u * b.w);
        float v = dot4(ns, c);
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        if (row < p.dv) {
            __stcs(reinterpret_cast<float4 *>(So + (size_t)row * DK + col), ns);
            if (lane % LPR == 0) p.y[(size_t)nh * p.dv + row] = from_f32<T>(fmaf(dh, x, v));
        }
    }
}

// carried inputs of the b and c channels, in place: out of the step kernel's way
template <typename T>
__global__ void __launch_bounds__(256)
move_bc_kernel(const T *xbc, T *cs, int64_t row, size_t C, int first, int W) {
    const int ch = first + blockIdx.y * 256 + threadIdx.x, n = blockIdx.x;
    if (ch >= (int)C) return;
    T *p = cs + (size_t)n * (W - 1) * C + ch;
    for (int m = 0; m < W - 2; ++m) p[m * C] = p[(m + 1) * C];
    p[(size_t)(W - 2) * C] = xbc[(int64_t)n * row + ch];
}

template <int DK, typename T>
cudaError_t launch_dk(const SsmStepArgs &a, cudaStream_t stream) {
    const bool conv = a.conv_w != nullptr;
    const bool in_place = conv && a.conv_state == a.conv_state_out;
    StepParams<T> p{static_cast<const T *>(a.xbc), a.dt, a.a, a.d, a.dt_bias, a.conv_w, a.conv_b,
                    static_cast<const T *>(a.conv_state), static_cast<T *>(a.conv_state_out), a.state,
                    a.state_out, static_cast<T *>(a.y), a.HK, a.HV, a.dv, conv ? a.conv_width : 0,
                    a.xbc_row, a.conv_silu, a.softplus, conv && !in_place};
    constexpr int NB = 8, BAND = kWarps * (32 / (DK / 4)) * NB;
    const dim3 grid((unsigned)(a.N * a.HV), (unsigned)((a.dv + BAND - 1) / BAND));
    ssm_step_kernel<DK, NB, T><<<grid, kWarps * 32, 0, stream>>>(p);
    if (in_place) {
        const int first = a.HV * a.dv, bc = 2 * a.HK * DK;
        move_bc_kernel<T><<<dim3((unsigned)a.N, (unsigned)((bc + 255) / 256)), 256, 0, stream>>>(
            p.xbc, p.cs_out, a.xbc_row, (size_t)first + bc, first, a.conv_width);
    }
    return cudaGetLastError();
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

cudaError_t launch_ssm_step(const SsmStepArgs &a, cudaStream_t stream) {
    return a.dtype == GDN_BF16 ? launch_typed<__nv_bfloat16>(a, stream) : launch_typed<float>(a, stream);
}

}  // namespace gdn
