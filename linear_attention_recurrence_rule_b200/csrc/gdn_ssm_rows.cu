// Selective state space scan on CUDA cores: fp32 calls and the head dims that
// the tensor-core scan does not take.
//
//   delta_t = softplus(dt_t + bias_h) (or dt_t + bias_h),  alpha_t = exp(delta_t a_h)
//   S_t = alpha_t S_{t-1} + delta_t x_t b_t^T,   y_t = S_t c_t + d_h x_t
//
// The rows of a state (one per value) never mix, so a warp walks the tokens with
// its rows in registers: a thread holds 8 rows x 8 columns, DK/8 lanes a row.  A
// token costs a lane 64 multiplies and 64 multiply-adds for the update and 64 for the
// read-out, done on packed fp32 pairs: the instructions issued are what bounds the
// kernel, so a thread's tile is as large as its registers take (7 shared loads a token
// for 64 elements; 4 rows took 3.0 instructions per element, 8 take 2.3), and the sums
// of two tokens x 8 rows are reduced together, transposed (15 shuffles for 16 sums).
// Tokens come in tiles of 16 by cp.async, one tile ahead.
//
// What bounds it is the fp32 multiply-add rate (packed pairs save instructions, not
// rate), so a tile whose decays multiply to no less than 2^-60 -- nearly every one -- is
// run on the state divided by its decays since the tile's start: with
// Gamma_t = alpha_1 .. alpha_t,  S'_t = S'_{t-1} + (delta_t / Gamma_t) x_t b_t^T  and
// y_t = Gamma_t S'_t c_t + d x_t, two operations per element and token instead of three,
// and one instead of two in the first pass; the state is multiplied by the tile's decay
// once at its end.  Nothing overflows within 2^60, and a sum keeps its relative accuracy
// whatever it is divided by.  Stronger tiles take the plain form.
//
// As far into a tile as the log decays add up to less than 1/4, Gamma is the exponential of
// the sum, one rounding a tile and not one a token: a product of 1000 decays near 1, each
// rounded by up to 2^-25, is off by up to 3e-5, all in one direction where the step sizes
// repeat.  What a tile's decay was rounded by goes into the next tile's log, so the product of
// all of them stays within two roundings of the exact one (8192 equal tokens, log decays of 0.5
// to 1.5 in all: states off by 4.3e-4 at worst, now 3.2e-6, their own roundings).  Farther on
// Gamma is the product of the tokens' decays, whose errors neighbours share (a sum of 40 has few
// digits left for the differences); such states do not live to gather many roundings.  y of 2048
// tokens with 32 heads of 128 (relative norm): 1.6e-7 to 9.1e-7, now 1.2e-7 to 1.4e-7, in the
// same time (235 us, 236 us).  A tile's Gammas stand between it and the one before: the sum and
// the product are scanned side by side, and 1 / Gamma is taken by the reciprocal (a division:
// 2 heads of 32 18.1 us for 17.1, 16K tokens of 32 heads of 32 298 us for 272).
//
// The tokens of a segment follow one another, so one segment per sequence would
// leave most SMs without work.  The sequence is cut into segments (find_seg): a
// first pass forms each segment's own state from zero and its decay, combine_kernel
// chains them, and the second pass runs every segment from its start state.
#include <type_traits>

#include "gdn_ssm_common.cuh"

namespace gdn {
namespace ssm {

constexpr int kTile = 16;        // tokens per tile
constexpr int kCols = 8;         // state columns per thread
constexpr float kMildTile = 0x1p-60f;
constexpr float kNearOne = 0.25f;

struct RowParams {
    const void *x, *b, *c;
    const float *dt, *a, *d, *dt_bias;
    int64_t x_row, b_row, c_row;
    int HK, HV, dv;
    bool softplus;
    void *y;
    float *hT;               // null: not wanted
    const float *h0;         // null: zero
    float *seg_state;        // [segments][HV][dv][dk]: own states (first pass), start states (second)
    float *seg_decay;        // [segments][HV]
    bool chained;            // the slots hold every segment's start state (hT may then alias h0)
    SegMap map;
};

__device__ __forceinline__ void cp16(void *dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)),
                 "l"(src)
                 : "memory");
}

// a thread's 8 columns: two float4 half a row apart (fp32: conflict-free 16-byte
// reads) or 8 consecutive ones (bf16: one 16-byte read)
template <int DK, typename T>
__device__ __forceinline__ int col_of(int lane_in_row, int quad) {
    return sizeof(T) == 4 ? quad * (DK / 2) + 4 * lane_in_row : 8 * lane_in_row + 4 * quad;
}
__device__ __forceinline__ void load_cols(const float *row, int l, int dk, float2 (&v)[4]) {
    const float4 p = *reinterpret_cast<const float4 *>(row + 4 * l);
    const float4 q = *reinterpret_cast<const float4 *>(row + dk / 2 + 4 * l);
    v[0] = make_float2(p.x, p.y);
    v[1] = make_float2(p.z, p.w);
    v[2] = make_float2(q.x, q.y);
    v[3] = make_float2(q.z, q.w);
}
__device__ __forceinline__ void load_cols(const __nv_bfloat16 *row, int l, int, float2 (&v)[4]) {
    const uint4 u = *reinterpret_cast<const uint4 *>(row + 8 * l);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        v[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    unsigned long long ua, ub, ud;
    memcpy(&ua, &a, 8);
    memcpy(&ub, &b, 8);
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(ud) : "l"(ua), "l"(ub));
    float2 d;
    memcpy(&d, &ud, 8);
    return d;
}

// e^x - 1 for |x| < kNearOne: its Taylor series, cut off below 2^-29 of the sum
__device__ __forceinline__ float near_expm1(float x) {
    const float x2 = x * x;
    float hi = fmaf(1.f / 5040.f, x, 1.f / 720.f);
    hi = fmaf(hi, x2, fmaf(1.f / 120.f, x, 1.f / 24.f));
    const float lo = fmaf(1.f / 6.f, x, 0.5f);
    return fmaf(x2, fmaf(hi, x2, lo), x);
}

// ROWS state rows per thread: 8 (4 where a warp of 8 would have more rows than the head), or
// 2 where there is too little to do to fill the SMs and a token's latency counts
template <int DK, int ROWS>
__host__ __device__ constexpr int rows_per_warp() { return 32 / (DK / kCols) * ROWS; }

// v[N] summed over the W lanes of a row group: halves the values while it halves the
// lanes.  `first`: the index of the value now in v[0] (then v[1], ... follow it).
template <int N, int W>
__device__ __forceinline__ void reduce(float *v, int lane, int &first) {
    if constexpr (W > 1) {
        if constexpr (N > 1) {
            const bool up = (lane & (W / 2)) != 0;
#pragma unroll
            for (int i = 0; i < N / 2; ++i) {
                const float keep = up ? v[N / 2 + i] : v[i], send = up ? v[i] : v[N / 2 + i];
                v[i] = keep + __shfl_xor_sync(0xffffffffu, send, W / 2);
            }
            if (up) first += N / 2;
            reduce<N / 2, W / 2>(v, lane, first);
        } else {
            v[0] += __shfl_xor_sync(0xffffffffu, v[0], W / 2);
            reduce<1, W / 2>(v, lane, first);
        }
    }
}

// one tile of raw tokens (16-byte copies and reads: so is the second tile's start)
template <int DK, typename T>
struct alignas(16) Tile {
    T b[kTile][DK];
    T c[kTile][DK];
    T x[kTile][128];
    float2 step[kTile];     // delta_t / Gamma_t, Gamma_t (mild) or delta_t, alpha_t
    float total;            // the tile's decay where it is mild, else 0
};

// READ: the second pass (start states, read-out, final state); otherwise the first
// CTAs per SM: 8 rows fill 128 registers and still gain from a fourth CTA (3: 240 -> 252 us for
// the layer); 4 and 2 rows come where there are fewer CTAs, and spills cost more than another
// CTA gains (4 rows, 16 x 300 tokens of 64 heads of 32: 7 CTAs 107 us, 5 82 us; 2 rows, 4096
// tokens of 64 heads of 32: 8 CTAs 158 us, 7 145 us, 5 158 us)
template <int DK, int ROWS, typename T, bool READ>
__global__ void __launch_bounds__(128, ROWS == 8 ? 4 : ROWS == 4 ? 5 : 7)
scan_rows_kernel(const RowParams p) {
    constexpr int LPR = DK / kCols;          // lanes per row group
    constexpr int RPW = rows_per_warp<DK, ROWS>();
    constexpr int AT_ONCE = ROWS == 2 ? 4 : 2;   // tokens whose sums are reduced together
    constexpr int V = 16 / (int)sizeof(T);   // elements per 16 bytes
    extern __shared__ __align__(16) uint8_t raw[];
    Tile<DK, T> *tiles = reinterpret_cast<Tile<DK, T> *>(raw);
    const int nt = blockDim.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rpc = (nt >> 5) * RPW;         // rows per CTA
    const int bands = p.dv / rpc;
    int slot = blockIdx.x / (p.HV * bands);
    const int hb = blockIdx.x - slot * (p.HV * bands);
    if (READ) wait_for_previous();
    else let_next_start();
    const Seg seg = find_seg(p.map, slot);
    if (!seg.ok) return;
    if (!READ && seg.last) return;           // nothing follows: its own state is not needed
    const int h = hb / bands, row0 = (hb - h * bands) * rpc;
    const int ck = h / (p.HV / p.HK);
    const int l = lane % LPR, grp = lane / LPR;
    const int lrow = warp * RPW + grp * ROWS;        // first row of this thread in the CTA
    const T *xp = static_cast<const T *>(p.x) + seg.t0 * p.x_row + (int64_t)h * p.dv + row0;
    const T *bp = static_cast<const T *>(p.b) + seg.t0 * p.b_row + (int64_t)ck * DK;
    const T *cp = static_cast<const T *>(p.c) + seg.t0 * p.c_row + (int64_t)ck * DK;
    const float *dtp = p.dt + seg.t0 * p.HV + h;
    const float ah = p.a[h], bias = p.dt_bias ? p.dt_bias[h] : 0.f;
    const float dh = READ && p.d ? p.d[h] : 0.f;
    const size_t st = ((size_t)slot * p.HV + h) * p.dv * DK;      // this segment's slot
    const size_t sq = ((size_t)seg.n * p.HV + h) * p.dv * DK;           // this sequence's state

    float2 S[ROWS][4];
    const float *src = nullptr;
    if (READ) src = p.chained ? p.seg_state + st : p.h0 ? p.h0 + sq : nullptr;
#pragma unroll
    for (int r = 0; r < ROWS; ++r)
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
            if (src) f = *reinterpret_cast<const float4 *>(src + (size_t)(row0 + lrow + r) * DK + col_of<DK, T>(l, q));
            S[r][2 * q] = make_float2(f.x, f.y);
            S[r][2 * q + 1] = make_float2(f.z, f.w);
        }

    const int ntiles = (seg.len + kTile - 1) / kTile;
    // dt of the tile that is issued next (warp 0): loaded a tile ahead, so that its trip
    // to memory does not stand between a tile and the one before it
    auto load_dt = [&](int k) {
        const int64_t t = (int64_t)k * kTile + lane;
        return warp == 0 && lane < kTile && t < seg.len ? dtp[t * p.HV] : 0.f;
    };
    float ahead = load_dt(0);
    float left = 0.f;        // log of the decay so far over what the states were multiplied by
    double run = 0.;         // sum of all log decays
    auto issue = [&](int k) {
        if (k < ntiles) {
            Tile<DK, T> &t = tiles[k & 1];
            const int64_t at = (int64_t)k * kTile;
            const int m = min(kTile, seg.len - k * kTile);
            for (int i = tid; i < m * (DK / V); i += nt) {
                const int r = i / (DK / V), e = (i - r * (DK / V)) * V;
                cp16(&t.b[r][e], bp + (at + r) * p.b_row + e);
                if (READ) cp16(&t.c[r][e], cp + (at + r) * p.c_row + e);
            }
            const int xv = rpc / V;
            for (int i = tid; i < m * xv; i += nt) {
                const int r = i / xv, e = (i - r * xv) * V;
                cp16(&t.x[r][e], xp + (at + r) * p.x_row + e);
            }
            if (warp == 0) {
                const bool in = lane < m;
                const float dl = in ? step_size(ahead, bias, p.softplus) : 0.f;
                ahead = load_dt(k + 1);
                const float g = in ? dl * ah : 0.f, al = expf(g);
                float sum = g, gamma = al;
#pragma unroll
                for (int off = 1; off < kTile; off <<= 1) {
                    const float v = __shfl_up_sync(0xffffffffu, sum, off), w = __shfl_up_sync(0xffffffffu, gamma, off);
                    if (lane >= off) {
                        sum += v;
                        gamma *= w;
                    }
                }
                if (!READ) run += (double)__shfl_sync(0xffffffffu, sum, kTile - 1);
                const float lg = sum + left, less = near_expm1(lg);
                const bool near = fabsf(lg) < kNearOne;
                gamma = near ? 1.f + less : gamma;
                const float total = __shfl_sync(0xffffffffu, gamma, kTile - 1);
                // what 1 + less was rounded by (exact, |less| < 1); 1 / gamma is near enough 1 - less
                left = __shfl_sync(0xffffffffu, near ? ((1.f - gamma) + less) * (1.f - less) : 0.f, kTile - 1);
                const bool mild = total >= kMildTile;
                const float2 step = mild ? make_float2(dl * __frcp_rn(gamma), gamma) : make_float2(dl, al);
                if (lane < kTile) t.step[lane] = step;
                if (lane == 0) t.total = mild ? total : 0.f;
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    issue(0);
    for (int k = 0; k < ntiles; ++k) {
        issue(k + 1);
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        __syncthreads();
        const Tile<DK, T> &t = tiles[k & 1];
        const int m = min(kTile, seg.len - k * kTile);
        T *yo = READ ? static_cast<T *>(p.y) + ((seg.t0 + (int64_t)k * kTile) * p.HV + h) * p.dv + row0 : nullptr;
        // U tokens from token i
        auto tokens = [&](auto count, auto kind, int i) {
            constexpr int U = decltype(count)::value;
            constexpr bool MILD = decltype(kind)::value;
            float acc[U * ROWS], xr[U * ROWS];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float2 bb[4], cc[4];
                load_cols(t.b[i + u], l, DK, bb);
                if (READ) load_cols(t.c[i + u], l, DK, cc);
                const float2 step = t.step[i + u];
                const float2 al2 = make_float2(step.y, step.y);
                if constexpr (ROWS >= 4) {
#pragma unroll
                    for (int r = 0; r < ROWS; r += 4) {
                        const float4 f = load4(&t.x[i + u][lrow + r]);
                        xr[u * ROWS + r] = f.x;
                        xr[u * ROWS + r + 1] = f.y;
                        xr[u * ROWS + r + 2] = f.z;
                        xr[u * ROWS + r + 3] = f.w;
                    }
                } else {
#pragma unroll
                    for (int r = 0; r < ROWS; ++r) xr[u * ROWS + r] = to_f32(t.x[i + u][lrow + r]);
                }
#pragma unroll
                for (int r = 0; r < ROWS; ++r) {
                    const float w = step.x * xr[u * ROWS + r];
                    const float2 w2 = make_float2(w, w);
#pragma unroll
                    for (int j = 0; j < 4; ++j) S[r][j] = MILD ? fma2(w2, bb[j], S[r][j]) : fma2(S[r][j], al2, mul2(w2, bb[j]));
                    if (READ) {
                        float2 s2 = mul2(S[r][0], cc[0]);
#pragma unroll
                        for (int j = 1; j < 4; ++j) s2 = fma2(S[r][j], cc[j], s2);
                        acc[u * ROWS + r] = s2.x + s2.y;
                    }
                }
            }
            if (READ) {
                int first = 0;
                reduce<U * ROWS, LPR>(acc, lane, first);
                // values left per lane; fewer values than lanes: the lanes with low bits 0 write
                constexpr int M = U * ROWS / LPR > 0 ? U * ROWS / LPR : 1;
                constexpr int IDLE = LPR / (U * ROWS) > 0 ? LPR / (U * ROWS) : 1;
                if ((lane & (IDLE - 1)) == 0) {
#pragma unroll
                    for (int q = 0; q < M; ++q) {
                        const int id = first + q, u = id / ROWS, r = id % ROWS;
                        const float xv = to_f32(t.x[i + u][lrow + r]);
                        const float v = MILD ? acc[q] * t.step[i + u].y : acc[q];
                        yo[(int64_t)(i + u) * p.HV * p.dv + lrow + r] = from_f32<T>(fmaf(dh, xv, v));
                    }
                }
            }
        };
        auto tile = [&](auto kind) {
            int i = 0;
#pragma unroll 1
            for (; i + AT_ONCE <= m; i += AT_ONCE) tokens(std::integral_constant<int, AT_ONCE>{}, kind, i);
#pragma unroll 1
            for (; i < m; ++i) tokens(std::integral_constant<int, 1>{}, kind, i);
        };
        const float total = t.total;
        if (total > 0.f) {
            tile(std::true_type{});
            const float2 t2 = make_float2(total, total);
#pragma unroll
            for (int r = 0; r < ROWS; ++r)
#pragma unroll
                for (int j = 0; j < 4; ++j) S[r][j] = mul2(S[r][j], t2);
        } else {
            tile(std::false_type{});
        }
        __syncthreads();
    }
    float *dst = READ ? (seg.last && p.hT ? p.hT + sq : nullptr) : p.seg_state + st;
    if (dst) {
#pragma unroll
        for (int r = 0; r < ROWS; ++r)
#pragma unroll
            for (int q = 0; q < 2; ++q)
                *reinterpret_cast<float4 *>(dst + (size_t)(row0 + lrow + r) * DK + col_of<DK, T>(l, q)) =
                    make_float4(S[r][2 * q].x, S[r][2 * q].y, S[r][2 * q + 1].x, S[r][2 * q + 1].y);
    }
    if (!READ && row0 == 0 && tid == 0) p.seg_decay[(size_t)slot * p.HV + h] = expf((float)run);
}

// Chains the segments of each sequence and head: slot i is read as segment i's own
// state and overwritten with its start state; the state behind the last segment
// goes to hT where `whole` (then the last segment's own state is there too).
// One thread per 4 elements.  The slots are read in batches of 8 ahead of their
// overwriting, so that a batch costs one trip to L2 and not eight (64K tokens, 9
// segments of 32 states of 128 x 128, cold: 42 us -> 21 us).
constexpr int kChain = 8;
__global__ void __launch_bounds__(256)
combine_kernel(float *seg_state, const float *seg_decay, const float *h0, float *hT, int HV, int elems,
               bool whole, const SegMap map) {
    let_next_start();
    const int e = (blockIdx.y * 256 + threadIdx.x) * 4;
    const int n = blockIdx.x / HV, h = blockIdx.x - n * HV;
    const size_t sq = ((size_t)n * HV + h) * elems + e;
    float4 S = make_float4(0.f, 0.f, 0.f, 0.f);
    if (h0 && e < elems) S = *reinterpret_cast<const float4 *>(h0 + sq);
    wait_for_previous();
    if (e >= elems) return;
    const int s0 = map.table ? map.first[n] : n * map.nseg;
    const int s1 = map.table ? map.first[n + 1] : s0 + map.nseg;
    const int end = whole ? s1 : s1 - 1;
    const size_t step = (size_t)HV * elems;
    float4 *slot = reinterpret_cast<float4 *>(seg_state + ((size_t)s0 * HV + h) * elems + e);
    const float *decay = seg_decay + (size_t)s0 * HV + h;
    for (int s = s0; s < end; s += kChain) {
        const int m = min(kChain, end - s);
        float4 own[kChain];
        float g[kChain];
#pragma unroll
        for (int i = 0; i < kChain; ++i)
            if (i < m) {
                own[i] = __ldcg(slot + i * (step / 4));
                g[i] = __ldcg(decay + i * HV);
            }
#pragma unroll
        for (int i = 0; i < kChain; ++i)
            if (i < m) {
                slot[i * (step / 4)] = S;
                S = make_float4(fmaf(g[i], S.x, own[i].x), fmaf(g[i], S.y, own[i].y), fmaf(g[i], S.z, own[i].z),
                                fmaf(g[i], S.w, own[i].w));
            }
        slot += m * (step / 4);
        decay += m * HV;
    }
    if (whole) {
        if (hT) *reinterpret_cast<float4 *>(hT + sq) = S;
    } else {
        *slot = S;
    }
}

// Segment table of a packed batch: one block, a running sum over tiles of 1024 sequences.
// With `order` also the segments by falling length (each counts those before it): CTAs
// take their work in the order of their indexes, and a long segment that starts behind
// short ones is waited for by all (8 prompts of 0 to 12288 tokens, 32 heads of 64: the
// schedule 40 -> 32 chunks long, the call 246 -> 200 to 208 us).
__global__ void __launch_bounds__(1024)
plan_kernel(const int32_t *cu, int N, int seg_len, int bound, int4 *table, int *first, int *order) {
    __shared__ int part[32];
    __shared__ int base;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) base = 0;
    __syncthreads();
    for (int n0 = 0; n0 < N; n0 += 1024) {
        const int n = n0 + tid;
        int t0 = 0, len = 0, cnt = 0;
        if (n < N) {
            t0 = cu[n];
            len = cu[n + 1] - t0;
            cnt = len > 0 ? (len - 1) / seg_len + 1 : 1;
        }
        int inc = cnt;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, inc, off);
            if (lane >= off) inc += y;
        }
        if (lane == 31) part[warp] = inc;
        __syncthreads();
        if (warp == 0) {
            int q = part[lane];
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, q, off);
                if (lane >= off) q += y;
            }
            part[lane] = q;
        }
        __syncthreads();
        const int at = base + inc - cnt + (warp ? part[warp - 1] : 0);
        if (n < N) {
            first[n] = at;
            for (int i = 0; i < cnt && at + i < bound; ++i)
                table[at + i] = make_int4(n, t0 + i * seg_len, min(seg_len, len - i * seg_len), i);
        }
        __syncthreads();
        if (tid == 1023) base = at + cnt;
        __syncthreads();
    }
    if (tid == 0) first[N] = base;
    if (!order) return;
    __shared__ int lens[kOrdered];
    static_assert(kOrdered == 1024, "a thread per segment");
    const int total = min(base, bound), mine = tid < total ? table[tid].z : -1;
    lens[tid] = mine;
    __syncthreads();
    int at = 0;
    for (int s = 0; s < total; ++s) at += lens[s] > mine || (lens[s] == mine && s < tid);
    if (tid < bound) order[tid < total ? at : tid] = tid;
}

cudaError_t launch_plan(const int32_t *cu, int N, int seg_len, int bound, int4 *table, int *first, int *order,
                        cudaStream_t stream) {
    plan_kernel<<<1, 1024, 0, stream>>>(cu, N, seg_len, bound, table, first, order);
    return cudaGetLastError();
}
cudaError_t launch_combine(float *seg_state, const float *seg_decay, const float *h0, float *hT, int N, int HV, int elems,
                           bool whole, const SegMap &map, cudaStream_t stream) {
    const dim3 grid((unsigned)((int64_t)N * HV), (elems / 4 + 255) / 256);
    return launch_after(combine_kernel, grid, dim3(256), 0, stream, seg_state, seg_decay, h0, hT, HV, elems, whole, map);
}

// ---- host: how the call is cut ----
struct Cut {
    int seg_len, nseg;      // tokens per segment; segments per sequence (without cu_seqlens)
    int bound;              // segments at most, over all sequences
    bool used;              // the call needs its workspace
    size_t table, first, order, decay, state, total;   // byte offsets in the workspace
};

// warps per CTA of a head with `rows` rows per thread
static int warps_of(int dk, int dv, int rows) { return min(4, dv / (32 / (dk / kCols) * rows)); }
static int full_rows(int dk, int dv) { return 32 / (dk / kCols) * 8 <= dv ? 8 : 4; }
static int ctas_per_state(const SsmArgs &a) {
    const int rows = full_rows(a.dk, a.dv);
    return a.dv / (warps_of(a.dk, a.dv, rows) * 32 / (a.dk / kCols) * rows);
}

// Segments are worth their first pass (half of the second's arithmetic) while the SMs have
// fewer than about 4 CTAs of 4 warps each without them; below 128 tokens a segment's start
// and end states weigh as much as its tokens.  The workspace has room for what any call of as
// many sequences and tokens may take: their segments come to 592 CTAs at most, or are one a
// sequence.
static Cut cut_rows(const SsmArgs &a) {
    Cut c{};
    const bool packed = a.cu_seqlens != nullptr;
    const int64_t longest = a.T > 0 ? a.T : 1;
    const int64_t head = (int64_t)a.HV * ctas_per_state(a), base = head * (packed ? 1 : a.N);
    int64_t nseg = base >= 592 ? 1 : 592 / base;
    int64_t len = (longest + nseg - 1) / nseg;
    len = (len + kTile - 1) / kTile * kTile;
    if (len < 128) len = 128;
    if (len > (1 << 30)) len = 1 << 30;
    c.seg_len = (int)len;
    c.nseg = (int)((longest + len - 1) / len);
    // (a sequence of l > 0 tokens has 1 + (l - 1) / seg_len segments)
    const int64_t bound = packed ? (int64_t)a.N + c.nseg - 1 : (int64_t)a.N * c.nseg;
    c.bound = bound * a.HV * 4 > 0x7fffffff ? -1 : (int)bound;   // grid.x
    c.used = packed || c.nseg > 1;
    const int64_t parts = (longest + 127) / 128, most = 592 / head > 1 ? 592 / head : 1;
    int64_t slots = packed ? a.N + min(most, parts) - 1 : max((int64_t)a.N, min(most, a.N * parts));
    if (slots < bound) slots = bound;    // (more than 2^30 tokens in a sequence)
    auto up = [](size_t v) { return (v + 255) & ~size_t(255); };
    size_t off = 256;
    c.table = off;
    if (packed) off += up((size_t)slots * sizeof(int4));
    c.first = off;
    if (packed) off += up((size_t)(a.N + 1) * sizeof(int));
    c.order = off;
    if (packed) off += up((size_t)min(slots, (int64_t)kOrdered) * sizeof(int));
    c.decay = off;
    off += up((size_t)slots * a.HV * sizeof(float));
    c.state = off;
    off += (size_t)slots * a.HV * a.dv * a.dk * sizeof(float);
    // (one segment a sequence, in every smaller call too: nothing is kept between kernels)
    c.total = packed || (most > 1 && parts > 1) ? off : 0;
    return c;
}

template <int DK, int ROWS, typename T>
static cudaError_t launch_rows_of(const SsmArgs &a, cudaStream_t stream) {
    const Cut cut = cut_rows(a);
    if (cut.bound < 0) return cudaErrorInvalidValue;
    cudaError_t err = cudaSuccess;
    uint8_t *ws = static_cast<uint8_t *>(a.workspace);
    const bool packed = a.cu_seqlens != nullptr;
    RowParams p{a.x, a.b, a.c, a.dt, a.a, a.d, a.dt_bias, a.x_row, a.b_row, a.c_row, a.HK, a.HV, a.dv,
                a.softplus, a.y, a.hT, a.h0, nullptr, nullptr, false,
                SegMap{nullptr, nullptr, a.N, cut.nseg, a.T, cut.seg_len}};
    if (cut.total && ws) {
        // the status word of gdn_read_status: nothing waits on the device here
        err = cudaMemsetAsync(ws, 0, sizeof(unsigned int), stream);
        if (err != cudaSuccess) return err;
    }
    if (cut.used) {
        p.seg_decay = reinterpret_cast<float *>(ws + cut.decay);
        p.seg_state = reinterpret_cast<float *>(ws + cut.state);
    }
    if (packed) {
        p.map.table = reinterpret_cast<int4 *>(ws + cut.table);
        p.map.first = reinterpret_cast<int *>(ws + cut.first);
        int *order = cut.bound <= kOrdered ? reinterpret_cast<int *>(ws + cut.order) : nullptr;
        p.map.order = order;
        err = launch_plan(a.cu_seqlens, a.N, cut.seg_len, cut.bound, reinterpret_cast<int4 *>(ws + cut.table),
                          reinterpret_cast<int *>(ws + cut.first), order, stream);
        if (err != cudaSuccess) return err;
    }
    const int warps = warps_of(DK, a.dv, ROWS);
    const dim3 block(32 * warps);
    const int bands = a.dv / (warps * rows_per_warp<DK, ROWS>());
    constexpr size_t smem = 2 * sizeof(Tile<DK, T>);
    static_assert(sizeof(Tile<DK, T>) % 16 == 0, "tile alignment");
    const dim3 grid((unsigned)((int64_t)cut.bound * a.HV * bands));
    const bool cuts = packed ? a.T > cut.seg_len : cut.nseg > 1;
    if (cuts) {
        p.chained = true;
        err = cudaFuncSetAttribute(scan_rows_kernel<DK, ROWS, T, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (err != cudaSuccess) return err;
        scan_rows_kernel<DK, ROWS, T, false><<<grid, block, smem, stream>>>(p);
        err = launch_combine(p.seg_state, p.seg_decay, a.h0, nullptr, a.N, a.HV, a.dv * DK, false, p.map, stream);
        if (err != cudaSuccess) return err;
    }
    err = cudaFuncSetAttribute(scan_rows_kernel<DK, ROWS, T, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (err != cudaSuccess) return err;
    if (cuts) return launch_after(scan_rows_kernel<DK, ROWS, T, true>, grid, block, smem, stream, p);
    scan_rows_kernel<DK, ROWS, T, true><<<grid, block, smem, stream>>>(p);
    return cudaGetLastError();
}

template <int DK, typename T>
static cudaError_t launch_rows(const SsmArgs &a, cudaStream_t stream) {
    // fewer than a warp per scheduler: 2 rows per thread (128 tokens, 2 heads of 32: 37 -> 21 us)
    const Cut cut = cut_rows(a);
    const int64_t warps = (int64_t)cut.bound * a.HV * ctas_per_state(a) * warps_of(DK, a.dv, full_rows(DK, a.dv));
    if (warps < 592) return launch_rows_of<DK, 2, T>(a, stream);
    if constexpr (DK == 32)
        if (full_rows(DK, a.dv) == 4) return launch_rows_of<DK, 4, T>(a, stream);
    return launch_rows_of<DK, 8, T>(a, stream);
}

}  // namespace ssm

bool ssm_supported(int dk, int dv) {
    return (dk == 32 || dk == 64 || dk == 128) && (dv == 32 || dv == 64 || dv == 128);
}

size_t ssm_workspace_bytes(const SsmArgs &a) {
    return ssm::tc_supported(a) ? ssm::tc_workspace_bytes(a) : ssm::cut_rows(a).total;
}
bool ssm_uses_workspace(const SsmArgs &a) { return ssm::tc_supported(a) || ssm::cut_rows(a).used; }

cudaError_t launch_ssm_prefill(const SsmArgs &a, cudaStream_t stream) {
    using namespace ssm;
    if (tc_supported(a)) return launch_tc(a, stream);
    const bool h = a.dtype == GDN_BF16;
    switch (a.dk) {
        case 32: return h ? launch_rows<32, __nv_bfloat16>(a, stream) : launch_rows<32, float>(a, stream);
        case 64: return h ? launch_rows<64, __nv_bfloat16>(a, stream) : launch_rows<64, float>(a, stream);
        default: return h ? launch_rows<128, __nv_bfloat16>(a, stream) : launch_rows<128, float>(a, stream);
    }
}

}  // namespace gdn
