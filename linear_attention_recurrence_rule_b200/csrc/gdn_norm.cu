// Norms around a block.
//
//   gated norm     y = rms(o) w f(z)   or   rms(o f(z)) w        over groups of D elements
//   residual norm  t = rms(x) wp f(z)  (norm and gate optional),
//                  h = residual + scale t,   y = rms(h) w
//   rms(u) = u / sqrt(mean(u^2) + eps),  f = sigmoid or SiLU,  w may stand for 1 + w
//
// Bound by memory: every element is read once, kept in registers as fp32 from the
// first sum of squares to the last product, and written once.  A row of D elements
// (16-byte vectors) belongs to 8, 16 or 32 lanes of a warp where it fits in their
// registers -- sums by shuffles, several rows per warp -- and to a whole block
// otherwise.  Rows that are not made of aligned 16-byte vectors (odd D, odd strides)
// take a kernel that reads element by element, three times at most, and so do rows of more
// than 4096 vectors (64 KB).  Alone and with a cold L2, of the measured copy rate: gated norm
// bf16 16384 x 2048 65%, 16384 x 2049 26%, 4096 groups of 32 x 100 6% (a block for each group
// of 100); residual norm with an fp32 residual, 16384 x 2048 94%, 16384 x 2049 66%, 2048 x
// 16384 62% (1024 threads leave 64 registers each, and the row's two fp32 copies spill), 512 x
// 65536 24%.
#include <type_traits>

#include "gdn_common.cuh"
#include "gdn_internal.h"

namespace gdn {
namespace {

template <typename T> struct Vec;
template <> struct Vec<__nv_bfloat16> {
    static constexpr int n = 8;
};
template <> struct Vec<float> {
    static constexpr int n = 4;
};

template <int N>
__device__ __forceinline__ void load_vec(const float *p, float (&f)[N]) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
        const float4 v = *reinterpret_cast<const float4 *>(p + i);
        f[i] = v.x;
        f[i + 1] = v.y;
        f[i + 2] = v.z;
        f[i + 3] = v.w;
    }
}
template <int N>
__device__ __forceinline__ void load_vec(const __nv_bfloat16 *p, float (&f)[N]) {
    static_assert(N == 8 || N == 4, "vector");
    uint32_t w[N / 2];
    if constexpr (N == 8) {
        const uint4 u = *reinterpret_cast<const uint4 *>(p);
        w[0] = u.x;
        w[1] = u.y;
        w[2] = u.z;
        w[3] = u.w;
    } else {
        const uint2 u = *reinterpret_cast<const uint2 *>(p);
        w[0] = u.x;
        w[1] = u.y;
    }
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
template <int N>
__device__ __forceinline__ void store_vec(float *p, const float (&f)[N]) {
#pragma unroll
    for (int i = 0; i < N; i += 4)
        *reinterpret_cast<float4 *>(p + i) = make_float4(f[i], f[i + 1], f[i + 2], f[i + 3]);
}
template <int N>
__device__ __forceinline__ void store_vec(__nv_bfloat16 *p, const float (&f)[N]) {
    uint32_t w[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    if constexpr (N == 8)
        *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    else
        *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
}

// the gate's factor: full precision for fp32 results, the hardware's exponential and
// reciprocal for bf16 ones (relative error about 1e-6 beside a rounding of 2^-8).  Four
// instructions for the sigmoid: with the layer steps' clamped division, 37 instructions an
// element kept a 4096 x 32 x 128 call from memory speed.
template <typename T>
__device__ __forceinline__ float gate_factor(float z, bool silu) {
    float s;
    if constexpr (sizeof(T) == 4) {
        s = gate_sigmoid(z);
    } else {
        float e;
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(-1.4426950408889634f * z));
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(1.f + e));
    }
    return silu ? z * s : s;
}

// sum over the TPR threads of a row; TPR > 32: the whole block
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float *part) {
#pragma unroll
    for (int o = (TPR > 32 ? 32 : TPR) / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (TPR > 32) {
        constexpr int NW = TPR > 32 ? TPR / 32 : 1;
        if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
        __syncthreads();
        v = 0.f;
#pragma unroll
        for (int i = 0; i < NW; ++i) v += part[i];
    }
    return v;
}

// (mean = ss / D as a product with 1 / D: one more rounding of 2^-24)
__device__ __forceinline__ float inv_rms(float ss, float inv_d, float eps) { return rsqrtf(fmaf(ss, inv_d, eps)); }

// Quotient by a divisor known on the host, exact for dividends below 2^31: with
// 2^(k-1) < d <= 2^k and m = ceil(2^(31+k) / d), q = n m / 2^(31+k).
struct Divisor {
    uint32_t m;
    int shift;
};
__device__ __forceinline__ uint32_t quotient(uint32_t n, const Divisor &d) {
    return (uint32_t)(((uint64_t)n * d.m) >> d.shift);
}
Divisor divisor(uint32_t d) {
    int k = 0;
    while (k < 31 && (1u << k) < d) ++k;
    return {(uint32_t)(((1ull << (31 + k)) + d - 1) / d), 31 + k};
}

constexpr int kSmallThreads = 256;   // block of the kernels with several rows per warp

// 16 bytes of one dtype, raw, as floats
template <typename T>
__device__ __forceinline__ void to_floats(const uint4 &u, float (&f)[Vec<T>::n]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(T) == 2) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        } else {
            f[i] = __uint_as_float(w[i]);
        }
    }
}

template <typename T, int TPR, int NV, bool FIRST>
__global__ void __launch_bounds__(TPR > 32 ? TPR : kSmallThreads)
gated_norm_kernel(const GatedNormArgs a, const Divisor groups, const float inv_d) {
    constexpr int VN = Vec<T>::n;
    constexpr int RPB = (TPR > 32 ? 1 : kSmallThreads / TPR);
    __shared__ float part[32];
    // (fewer than 2^31 groups: 32-bit indexes)
    const uint32_t unit = blockIdx.x * (uint32_t)RPB + (TPR > 32 ? 0 : threadIdx.x / TPR);
    const int lane = TPR > 32 ? threadIdx.x : threadIdx.x % TPR;
    const uint32_t G = (uint32_t)a.G;
    const bool live = unit < (uint32_t)(a.rows * a.G);
    const uint32_t r = live ? quotient(unit, groups) : 0u, g = live ? unit - r * G : 0u;
    const int64_t col = (int64_t)g * a.D;
    const T *o = static_cast<const T *>(a.o) + r * a.o_row + col;
    const T *z = static_cast<const T *>(a.z) + r * a.z_row + col;
    uint4 uo[NV], uz[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int e = (k * TPR + lane) * VN;
        if (live && e < a.D) {
            uo[k] = *reinterpret_cast<const uint4 *>(o + e);
            if (a.z) uz[k] = *reinterpret_cast<const uint4 *>(z + e);
        }
    }
    float u[NV][VN], f[NV][VN];
    float ss = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        if (live && (k * TPR + lane) * VN < a.D) {
            to_floats<T>(uo[k], u[k]);
            if (a.z) {
                to_floats<T>(uz[k], f[k]);
#pragma unroll
                for (int i = 0; i < VN; ++i) f[k][i] = gate_factor<T>(f[k][i], a.silu);
            } else {
#pragma unroll
                for (int i = 0; i < VN; ++i) f[k][i] = 1.f;
            }
#pragma unroll
            for (int i = 0; i < VN; ++i) {
                if (FIRST) u[k][i] *= f[k][i];
                ss = fmaf(u[k][i], u[k][i], ss);
            }
        }
    }
    const float inv = inv_rms(row_sum<TPR>(ss, part), inv_d, a.eps), one = a.unit_offset ? 1.f : 0.f;
    const float *w = a.weight ? a.weight + (a.weight_per_group ? col : 0) : nullptr;
    T *y = static_cast<T *>(a.y) + (int64_t)unit * a.D;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int e = (k * TPR + lane) * VN;
        if (live && e < a.D) {
            if (w) {
                float wv[VN];
                load_vec<VN>(w + e, wv);
#pragma unroll
                for (int i = 0; i < VN; ++i) u[k][i] *= inv * (wv[i] + one);
            } else {
#pragma unroll
                for (int i = 0; i < VN; ++i) u[k][i] *= inv;
            }
#pragma unroll
            for (int i = 0; i < VN; ++i)
                if (!FIRST) u[k][i] *= f[k][i];
            store_vec<VN>(y + e, u[k]);
        }
    }
}

template <typename T, typename TR, int TPR, int NV>
__global__ void __launch_bounds__(TPR > 32 ? TPR : kSmallThreads)
residual_norm_kernel(const ResidualNormArgs a, const float inv_c) {
    constexpr int VN = Vec<T>::n;
    constexpr int RPB = TPR > 32 ? 1 : kSmallThreads / TPR;
    __shared__ float part[2][32];
    const int64_t row = (int64_t)blockIdx.x * RPB + (TPR > 32 ? 0 : threadIdx.x / TPR);
    const int lane = TPR > 32 ? threadIdx.x : threadIdx.x % TPR;
    const bool live = row < a.rows;
    const int64_t at = live ? row * a.C : 0;
    const T *x = static_cast<const T *>(a.x) + at;
    const T *z = a.z ? static_cast<const T *>(a.z) + at : nullptr;
    const TR *res = a.residual ? static_cast<const TR *>(a.residual) + at : nullptr;
    float t[NV][VN], h[NV][VN];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int e = (k * TPR + lane) * VN;
        if (live && e < a.C) {
            load_vec<VN>(x + e, t[k]);
            if (res) load_vec<VN>(res + e, h[k]);
        }
    }
    if (a.post_weight) {
        float ss = 0.f;
#pragma unroll
        for (int k = 0; k < NV; ++k)
            if (live && (k * TPR + lane) * VN < a.C)
#pragma unroll
                for (int i = 0; i < VN; ++i) ss = fmaf(t[k][i], t[k][i], ss);
        const float inv = inv_rms(row_sum<TPR>(ss, part[0]), inv_c, a.eps);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int e = (k * TPR + lane) * VN;
            if (live && e < a.C) {
                float wv[VN];
                load_vec<VN>(a.post_weight + e, wv);
#pragma unroll
                for (int i = 0; i < VN; ++i) t[k][i] *= inv * (a.unit_offset ? 1.f + wv[i] : wv[i]);
            }
        }
    }
    float ss = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int e = (k * TPR + lane) * VN;
        if (live && e < a.C) {
            if (z) {
                float f[VN];
                load_vec<VN>(z + e, f);
#pragma unroll
                for (int i = 0; i < VN; ++i) t[k][i] *= gate_factor<T>(f[i], a.silu);
            }
#pragma unroll
            for (int i = 0; i < VN; ++i) {
                h[k][i] = res ? fmaf(a.scale, t[k][i], h[k][i]) : a.scale * t[k][i];
                ss = fmaf(h[k][i], h[k][i], ss);
            }
            if (a.residual_out) store_vec<VN>(static_cast<TR *>(a.residual_out) + at + e, h[k]);
        }
    }
    if (!a.y) return;
    const float inv = inv_rms(row_sum<TPR>(ss, part[1]), inv_c, a.eps);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int e = (k * TPR + lane) * VN;
        if (live && e < a.C) {
            float wv[VN];
            if (a.weight) load_vec<VN>(a.weight + e, wv);
#pragma unroll
            for (int i = 0; i < VN; ++i)
                h[k][i] *= inv * (a.weight ? (a.unit_offset ? 1.f + wv[i] : wv[i]) : 1.f);
            store_vec<VN>(static_cast<T *>(a.y) + at + e, h[k]);
        }
    }
}

// ---- rows that are not aligned 16-byte vectors: one block per row, element by element
constexpr int kOddThreads = 256;
__device__ __forceinline__ float block_sum(float v, float *part) {
    __syncthreads();   // an earlier sum's reads are over
    return row_sum<kOddThreads>(v, part);
}

template <typename T>
__global__ void __launch_bounds__(kOddThreads)
gated_norm_odd_kernel(const GatedNormArgs a) {
    __shared__ float part[32];
    const int64_t unit = blockIdx.x, r = unit / a.G;
    const int g = (int)(unit - r * a.G);
    const T *o = static_cast<const T *>(a.o) + r * a.o_row + (int64_t)g * a.D;
    const T *z = a.z ? static_cast<const T *>(a.z) + r * a.z_row + (int64_t)g * a.D : nullptr;
    T *y = static_cast<T *>(a.y) + (r * a.G + g) * a.D;
    float ss = 0.f;
    for (int e = threadIdx.x; e < a.D; e += kOddThreads) {
        float u = to_f32(o[e]);
        if (z && a.gate_first) u *= gate_factor<T>(to_f32(z[e]), a.silu);
        ss = fmaf(u, u, ss);
    }
    const float inv = inv_rms(block_sum(ss, part), 1.f / (float)a.D, a.eps);
    const float *w = a.weight ? a.weight + (a.weight_per_group ? (int64_t)g * a.D : 0) : nullptr;
    for (int e = threadIdx.x; e < a.D; e += kOddThreads) {
        float u = to_f32(o[e]);
        const float f = z ? gate_factor<T>(to_f32(z[e]), a.silu) : 1.f;
        if (a.gate_first) u *= f;
        u *= inv * (w ? (a.unit_offset ? 1.f + w[e] : w[e]) : 1.f);
        y[e] = from_f32<T>(a.gate_first ? u : u * f);
    }
}

template <typename T, typename TR>
__global__ void __launch_bounds__(kOddThreads)
residual_norm_odd_kernel(const ResidualNormArgs a) {
    __shared__ float part[32];
    const int64_t at = (int64_t)blockIdx.x * a.C;
    const T *x = static_cast<const T *>(a.x) + at;
    const T *z = a.z ? static_cast<const T *>(a.z) + at : nullptr;
    const TR *res = a.residual ? static_cast<const TR *>(a.residual) + at : nullptr;
    TR *ro = a.residual_out ? static_cast<TR *>(a.residual_out) + at : nullptr;
    T *y = a.y ? static_cast<T *>(a.y) + at : nullptr;
    float inv = 1.f;
    if (a.post_weight) {
        float ss = 0.f;
        for (int e = threadIdx.x; e < a.C; e += kOddThreads) {
            const float u = to_f32(x[e]);
            ss = fmaf(u, u, ss);
        }
        inv = inv_rms(block_sum(ss, part), 1.f / (float)a.C, a.eps);
    }
    auto h_of = [&](int e) {
        float t = to_f32(x[e]);
        if (a.post_weight) t *= inv * (a.unit_offset ? 1.f + a.post_weight[e] : a.post_weight[e]);
        if (z) t *= gate_factor<T>(to_f32(z[e]), a.silu);
        return res ? fmaf(a.scale, t, to_f32(res[e])) : a.scale * t;
    };
    float inv2 = 0.f;
    if (y) {
        float ss = 0.f;
        for (int e = threadIdx.x; e < a.C; e += kOddThreads) {
            const float h = h_of(e);
            ss = fmaf(h, h, ss);
        }
        inv2 = inv_rms(block_sum(ss, part), 1.f / (float)a.C, a.eps);
    }
    // residual_out may be the residual, y may be x: each element is read before it is written
    for (int e = threadIdx.x; e < a.C; e += kOddThreads) {
        const float h = h_of(e);
        if (ro) ro[e] = from_f32<TR>(h);
        if (y) y[e] = from_f32<T>(h * inv2 * (a.weight ? (a.unit_offset ? 1.f + a.weight[e] : a.weight[e]) : 1.f));
    }
}

bool vec_ok(const void *p, int64_t row, int elt) {
    return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && (row * elt) % 16 == 0;
}

// Threads per row and vectors per thread by the row's number of 16-byte vectors
template <typename F>
cudaError_t by_vectors(int nv, F f) {
    // (two vectors a thread from 9 on: what a thread does once weighs less per element)
    if (nv <= 8) return f(std::integral_constant<int, 8>{}, std::integral_constant<int, 1>{});
    if (nv <= 16) return f(std::integral_constant<int, 8>{}, std::integral_constant<int, 2>{});
    if (nv <= 32) return f(std::integral_constant<int, 16>{}, std::integral_constant<int, 2>{});
    if (nv <= 64) return f(std::integral_constant<int, 32>{}, std::integral_constant<int, 2>{});
    if (nv <= 128) return f(std::integral_constant<int, 128>{}, std::integral_constant<int, 1>{});
    if (nv <= 256) return f(std::integral_constant<int, 256>{}, std::integral_constant<int, 1>{});
    if (nv <= 512) return f(std::integral_constant<int, 256>{}, std::integral_constant<int, 2>{});
    if (nv <= 1024) return f(std::integral_constant<int, 256>{}, std::integral_constant<int, 4>{});
    if (nv <= 4096) return f(std::integral_constant<int, 1024>{}, std::integral_constant<int, 4>{});
    return cudaErrorInvalidValue;
}
int64_t blocks_of(int64_t rows, int tpr) {
    const int rpb = tpr > 32 ? 1 : kSmallThreads / tpr;
    return (rows + rpb - 1) / rpb;
}

template <typename T>
cudaError_t gated_norm(const GatedNormArgs &a, cudaStream_t stream) {
    constexpr int VN = Vec<T>::n;
    const int64_t units = a.rows * a.G;
    const bool vec = a.D % VN == 0 && a.D / VN <= 4096 && vec_ok(a.o, a.o_row, sizeof(T)) &&
                     vec_ok(a.z, a.z ? a.z_row : 0, sizeof(T)) && vec_ok(a.y, 0, 1) && vec_ok(a.weight, 0, 1);
    if (!vec) {
        gated_norm_odd_kernel<T><<<(unsigned)units, kOddThreads, 0, stream>>>(a);
        return cudaGetLastError();
    }
    return by_vectors(a.D / VN, [&](auto tpr, auto nv) {
        constexpr int TPR = decltype(tpr)::value, NV = decltype(nv)::value;
        auto kern = a.gate_first ? gated_norm_kernel<T, TPR, NV, true> : gated_norm_kernel<T, TPR, NV, false>;
        kern<<<(unsigned)blocks_of(units, TPR), TPR > 32 ? TPR : kSmallThreads, 0, stream>>>(a, divisor((uint32_t)a.G),
                                                                                           1.f / (float)a.D);
        return cudaGetLastError();
    });
}

template <typename T, typename TR>
cudaError_t residual_norm(const ResidualNormArgs &a, cudaStream_t stream) {
    constexpr int VN = Vec<T>::n;
    const bool vec = a.C % VN == 0 && a.C / VN <= 4096 && vec_ok(a.x, 0, 1) && vec_ok(a.z, 0, 1) &&
                     vec_ok(a.residual, 0, 1) && vec_ok(a.residual_out, 0, 1) && vec_ok(a.y, 0, 1) &&
                     vec_ok(a.post_weight, 0, 1) && vec_ok(a.weight, 0, 1);
    if (!vec) {
        residual_norm_odd_kernel<T, TR><<<(unsigned)a.rows, kOddThreads, 0, stream>>>(a);
        return cudaGetLastError();
    }
    return by_vectors(a.C / VN, [&](auto tpr, auto nv) {
        constexpr int TPR = decltype(tpr)::value, NV = decltype(nv)::value;
        residual_norm_kernel<T, TR, TPR, NV><<<(unsigned)blocks_of(a.rows, TPR),
                                               TPR > 32 ? TPR : kSmallThreads, 0, stream>>>(a, 1.f / (float)a.C);
        return cudaGetLastError();
    });
}

}  // namespace

cudaError_t launch_gated_norm(const GatedNormArgs &a, cudaStream_t stream) {
    return a.dtype == GDN_BF16 ? gated_norm<__nv_bfloat16>(a, stream) : gated_norm<float>(a, stream);
}

cudaError_t launch_residual_norm(const ResidualNormArgs &a, cudaStream_t stream) {
    if (a.dtype == GDN_F32) return residual_norm<float, float>(a, stream);
    return a.res_dtype == GDN_BF16 ? residual_norm<__nv_bfloat16, __nv_bfloat16>(a, stream)
                                   : residual_norm<__nv_bfloat16, float>(a, stream);
}

}  // namespace gdn
