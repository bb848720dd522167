// Selective state space scan on tensor cores: bf16 x, b, c with dk = 128 and value
// heads of 64 or 128, fp32 states and sums.
//
//   S_t = alpha_t S_{t-1} + delta_t x_t b_t^T,   y_t = S_t c_t + d x_t
//
// In chunks of 128 tokens, with G the chunk's running sum of log alpha:
//   y_i = e^{G_i} S_0 c_i + sum_{j<=i} P_ij x_j + d x_i,  P_ij = (c_i.b_j) e^{G_i-G_j} delta_j
//   S_1 = e^{G_L} S_0 + sum_j w_j x_j b_j^T,               w_j = e^{G_L-G_j} delta_j
// Nothing but the state ties the chunks, and the states add: a sequence is cut into
// segments, whose own states (from zero) are formed first, chained, and then every
// segment runs from its start state.  Three kernels:
//
//  * states_kernel, one CTA per (segment, value tile): S = sum_j (w_j x_j) b_j^T over
//    the whole segment with the decays to the segment's END in w_j (all <= delta_j, so
//    nothing overflows and nothing is rescaled on the way) -- one product with the
//    tokens as its inner dimension, chunk by chunk from the end.  w_j x_j is a full
//    fp32 value, so it enters as three bf16 terms (exactly): the states returned to the
//    caller carry fp32 accuracy.
//  * combine_kernel (gdn_ssm_rows.cu): chains the segments in place; hT.
//  * scan_kernel, one CTA per (segment, value tile), chunk by chunk: C B^T, the masked
//    and decayed P, C S^T, P X and the next state, all on tcgen05 with the state in
//    tensor memory.  Its state only feeds the bf16 y: P, w_j x_j and the S that is read out are
//    rounded to bf16, as the operands of its products, so a term of y inside its chunk is
//    rounded once on the way and one from before it twice.  y of the measured cases is off
//    by 1.83e-3 to 1.91e-3 in norm where the output's own rounding is 1.66e-3; the rest is
//    nearly all P's, a second product with P's remainder would take a quarter of the tensor
//    cores' time more and tensor memory that pairs of heads do not have.  (w_j in bf16 too, one
//    packed multiply for four instructions, was 1% faster, for a third rounding.)
//
// A value tile is 128 columns where it can be: one head of 128, or two heads of 64 of
// one group, which share C B^T and the loads of b and c; else one head of 64.
//
// scan_kernel keeps its state transposed, S^T [dk lanes][value columns].  Its warps: a
// loader (TMA), the MMA issuer, two for the tables (step sizes, running sums, the factors
// below; every other chunk each), and groups of four -- mask (C B^T -> P in the same
// tensor memory columns), state (S -> bf16 operand, S times e^{G_L}), weight (w x, in
// pieces of 32 tokens through a ring of 3) and output.  The mask takes e^{G_i-G_j} as the
// decays behind j in its 32-token block times those from there to i, both <= 1: one
// exponential per row and block.  On the diagonal a block whose log2 decays add up to no less
// than -100 has a common reference, its start (an exponential of a running sum over another
// one: off by up to 5e-5, beside the score's rounding to bf16 of 2^-8); stronger ones take one
// exponential per element.  All other sums of log decays run over the tokens between the two
// ends (block sums): a token that forgets everything (a log decay of thousands) would leave
// differences of running sums few digits for the tokens behind it.
//
// y leaves through the x tile: the output warps put their rows over the x they have read
// and TMA stores the tile (a part chunk is stored by the warps).  Their own stores, 32
// bytes a lane and a row apart, cost 15 to 80 us of the 64K case's 640 (the more, the
// lower the clock).
//
// What bounds it (64K tokens, 32 heads of 128, 16 groups: 1.62 GB, 247 us at the measured
// copy rate; 660 to 680 us in a long run, under the 1000 W cap): scan_kernel 369 us,
// states_kernel 203 us, combine_kernel 20 us, each alone.  scan_kernel takes about 5000 cycles
// per 128 tokens, and no one pipe fills them: the tensor cores read 224 KB of shared memory
// (1792 cycles at 128 bytes a cycle) and the schedulers issue 2400 instructions each (0.33 a
// cycle); taking any one role's shared memory accesses out changed the time by 5% at most, 13%
// fewer instructions by 0.5%.  What is left is the chain of one chunk: C S^T, the load of c
// into its one tile, C B^T, the mask, P X, the read-out, and beside it the state's way through
// the state warps and back.  Its order is a choice: C S^T waits for the read-out of the chunk
// before because y has two accumulators and tensor memory no second pair, and the tiles of b,
// c, x and P fill the 227 KB.  Measured and not kept: eight weight warps (640 ->
// 665 us), eight output or state warps (683 -> 700 us), a skip term from L2 instead of the
// shared x tile (740 -> 790 us), C S^T issued at whichever is ready first (565 -> 585 us),
// roles unrolled in full (they miss the instruction cache: 740 us against 410 us rolled),
// MMAs issued in rolled loops (95-130 cycles each instead of 64).
//
// Waits are bounded (about 2 s): a wait that gives up records GDN_ERR_TIMEOUT in the
// workspace's first word and every role winds down.
#include <cuda.h>

#include "gdn_ssm_common.cuh"
#include "gdn_tc_common.cuh"
#include "tc_primitives.cuh"
#include "tma_host.h"

namespace gdn {
namespace ssm {
namespace {

using namespace tc;
using namespace tcc;

constexpr int L = 128;      // tokens per chunk
constexpr int DK = 128;
constexpr float kLog2e = 1.4426950408889634f;

struct TcParams {
    const float *dt, *a, *d, *dt_bias, *h0;
    int HK, HV;
    bool soft;
    __nv_bfloat16 *y;
    float *seg_state, *seg_decay;
    unsigned int *status;
    bool chained;       // scan: start states from the slots (otherwise h0)
    bool whole;         // states: the last segment's state is wanted too
    int timeout_test;   // 1 (test only): the MMA warp issues nothing, as if its first wait had given up
    SegMap map;
};

constexpr long long kWaitCycles = 4000000000LL, kDrainCycles = 100000000LL;
// The roles' loops share the instruction cache, so what runs seldom is kept out of
// them: one copy of the polling loop.
__device__ __noinline__ bool wait_slow(uint64_t *bar, uint32_t parity, volatile int *abort_flag, unsigned int *status) {
    const long long t0 = clock64();
    for (;;) {
        if (__any_sync(0xffffffffu, *abort_flag != 0 || clock64() - t0 > kWaitCycles)) {
            *abort_flag = 1;
            atomicExch(status, (unsigned int)GDN_ERR_TIMEOUT);
            return false;
        }
        if (__all_sync(0xffffffffu, mbar_try_wait_sleep(bar, parity, 100000u))) return true;
    }
}
struct Waiter {
    uint64_t *bars;
    volatile int *abort_flag;
    unsigned int *status;
    // false once the CTA has given up (the same in every lane)
    __device__ __forceinline__ bool operator()(int b, uint32_t parity) const {
        if (__all_sync(0xffffffffu, mbar_try_wait(&bars[b], parity))) return true;
        return wait_slow(&bars[b], parity, abort_flag, status);
    }
    __device__ void drain(int b, uint32_t parity) const {
        const long long t0 = clock64();
        while (!mbar_try_wait(&bars[b], parity))
            if (clock64() - t0 > kDrainCycles) return;
    }
};

__device__ __forceinline__ void tma_prefetch_l2_2d(const CUtensorMap *map, int x, int y) {
    asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(x), "r"(y)
                 : "memory");
}
// 2-D tiled store from shared memory, tracked by the issuing thread's bulk group
__device__ __forceinline__ void tma_store_2d(const CUtensorMap *map, uint32_t src, int x, int y) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(src), "r"(x), "r"(y)
                 : "memory");
}
__device__ __forceinline__ void arrive(uint64_t *bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
// one arrival for the warp, after all its lanes
__device__ __forceinline__ void warp_arrive(uint64_t *bar) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) arrive(bar);
}
__device__ __forceinline__ uint64_t desc_add(uint64_t d, uint32_t bytes) { return d + (bytes >> 4); }
// hardware 2^x (relative error about 2^-22; -inf gives 0)
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ void tmem_ld32r(uint32_t taddr, float (&v)[32]) {
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, float (&v)[8]) {
    uint32_t r[8];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
    uint4 u;
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w) : "r"(addr));
    return u;
}
__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ float2 unpack2(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ float2 mulp(float2 a, float2 b) {
    unsigned long long ua, ub, ud;
    memcpy(&ua, &a, 8);
    memcpy(&ub, &b, 8);
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(ud) : "l"(ua), "l"(ub));
    float2 d;
    memcpy(&d, &ud, 8);
    return d;
}
__device__ __forceinline__ float2 subp(float2 a, float2 b) {
    unsigned long long ua, ub, ud;
    memcpy(&ua, &a, 8);
    memcpy(&ub, &b, 8);
    asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(ud) : "l"(ua), "l"(ub));
    float2 d;
    memcpy(&d, &ud, 8);
    return d;
}
// w x of a bf16 pair, rounded once
__device__ __forceinline__ uint32_t weighted(uint32_t x, float w) {
    const float2 f = mulp(unpack2(x), make_float2(w, w));
    return pack_bf16x2(f.x, f.y);
}

// One head's decay and step bias, a * log2 e and dt_bias.
struct HeadTab {
    float ah, bias;
};
// Step size and log2 decay of a token; no token: both 0.  A log2 decay below -150 is
// taken as -150: every factor with that token in it is 0 in fp32 either way, and the
// sums of the tokens around it keep their digits.
__device__ __forceinline__ float log_decay(float delta, float ah) { return fmaxf(delta * ah, -150.f); }
__device__ __forceinline__ void token_step(float dt, const HeadTab &t, bool in, bool soft, float &delta, float &g) {
    delta = in ? step_size(dt, t.bias, soft) : 0.f;
    g = in ? log_decay(delta, t.ah) : 0.f;
}
// Sums of g inside a 32-token block, a token per lane: `pre` up to and including the
// token, `suf` behind it; returns the block's sum.  Sums over longer spans add whole
// blocks to these, so no span's sum is a difference of larger ones.
__device__ __forceinline__ float block_sums(float g, int lane, float &pre, float &suf) {
    float up = g, down = g;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const float u = __shfl_up_sync(0xffffffffu, up, off), d = __shfl_down_sync(0xffffffffu, down, off);
        if (lane >= off) up += u;
        if (lane + off < 32) down += d;
    }
    pre = up;
    suf = __shfl_down_sync(0xffffffffu, down, 1);
    if (lane == 31) suf = 0.f;
    return __shfl_sync(0xffffffffu, down, 0);
}

// -------------------------------------------------------------------- segments' own states
// S[value][key] += (w x)^T b over the tokens of the segment.  The workers take x^T out of
// shared memory with transposing matrix loads, weight it and put it into tensor memory as
// three bf16 terms (the A operand, lanes = value columns): the products then read only b
// from shared memory (with the terms in shared memory it moved 384 KB per 128 tokens of a
// 128-wide tile instead of 192 KB, and took 280 us instead of 214 us for 64K tokens of 32
// heads of 128; 203 us now, its loads and stores there at 23% of their rate).  What bounds it:
// its 24 products a chunk take 1540 cycles, the workers' chain of a piece (load, split, store,
// signal) about as long again, and the two overlap in part; 0.47 of the issue slots are used.
// The first terms and the two small ones have an accumulator each, so that the small ones are not rounded
// away against the large sum, and every kFlush chunks both are added to sums in the
// workers' registers: the tensor cores truncate, and over the 456 additions of a 7K-token
// segment the sums fell short by 2.2e-6; over 64 by 3e-7.
template <int VT, int NH>
struct StatesCfg {
    static constexpr uint32_t XT = VT * 256;                 // x tile: 128 rows
    static constexpr uint32_t STAGE = 32768 + XT;            // b tile, x tile
    static constexpr int NS = 3;
    static constexpr uint32_t O_TAB = NS * STAGE;            // w to the 32-token block's end [NS][NH][128]
    static constexpr uint32_t O_SUM = O_TAB + NS * NH * 512; // the blocks' log2 decays [NS][NH][4]
    static constexpr uint32_t O_BAR = O_SUM + NS * NH * 16;
    static constexpr uint32_t BYTES = O_BAR + 256 + 1024;
};
static_assert(StatesCfg<128, 2>::BYTES <= 232448, "shared memory");
constexpr int kStTables = 4, kStTable0 = 2, kStWorkers = 16, kStWork0 = kStTable0 + kStTables, kStThreads = (kStWork0 + kStWorkers) * 32;
enum StBar { SB_F0, SB_E0 = SB_F0 + 3, SB_TF0 = SB_E0 + 3, SB_TE0 = SB_TF0 + 3, SB_WF0 = SB_TE0 + 3, SB_WE0 = SB_WF0 + 5,
             SB_DONE = SB_WE0 + 5, SB_READ, SB_END, SB_COUNT };
constexpr int kFlush = 8;   // chunks between two readings of the accumulators
// tensor memory: the sums of the first terms, of the small ones, a ring of pieces of 32
// tokens (three terms of 16 columns)
constexpr uint32_t TS_D = 0, TS_DS = 128, TS_A = 256, TS_PIECE = 48;
constexpr int kPieces = 5;

// four 8x8 blocks of 16-bit elements, each transposed over the warp; lane l gives the
// address of row l % 8 of block l / 8
__device__ __forceinline__ void ldsm_x4_t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
// 16 lanes x 8 columns: registers 2i, 2i + 1 hold columns 4i .. 4i + 3 of lanes l / 4 and
// l / 4 + 8 (column l % 4 of the four)
__device__ __forceinline__ void tmem_st_16x128b_x2(uint32_t taddr, const uint32_t (&w)[4]) {
    asm volatile("tcgen05.st.sync.aligned.16x128b.x2.b32 [%0], {%1,%2,%3,%4};" ::"r"(taddr), "r"(w[0]), "r"(w[1]),
                 "r"(w[2]), "r"(w[3])
                 : "memory");
}
// The upper halves of two floats as a bf16 pair (truncated), the floats' remainders left:
// a 24-bit significand is exactly three such parts.
__device__ __forceinline__ uint32_t high_pair(float2 x) {
    return __byte_perm(__float_as_uint(x.x), __float_as_uint(x.y), 0x7632);
}
__device__ __forceinline__ uint32_t take_high(float2 &x) {
    const uint32_t w = high_pair(x);
    x = subp(x, make_float2(__uint_as_float(__float_as_uint(x.x) & 0xffff0000u),
                            __uint_as_float(__float_as_uint(x.y) & 0xffff0000u)));
    return w;
}

template <int VT, int NH>
__global__ void __launch_bounds__(kStThreads, 1)
states_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_b, const TcParams p) {
    using Cfg = StatesCfg<VT, NH>;
    constexpr int DV = VT / NH;
    extern __shared__ uint8_t raw[];
    uint8_t *sm = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
    const uint32_t sb = smem_u32(sm);
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + Cfg::O_BAR);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(sm + Cfg::O_BAR + 8 * SB_COUNT);
    uint32_t *tslot = reinterpret_cast<uint32_t *>(sm + Cfg::O_BAR + 8 * SB_COUNT + 4);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tiles = p.HV / NH;
    int slot = blockIdx.x / tiles;
    const int head = (blockIdx.x - slot * tiles) * NH;
    let_next_start();
    // (no wait gives up within the first second)
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.status = 0u;
    const Seg seg = find_seg(p.map, slot);
    if (!seg.ok || (seg.last && !p.whole)) return;
    const int nch = (seg.len + L - 1) / L;
    if (threadIdx.x == 0) {
        for (int i = 0; i < 3; ++i) {
            mbar_init(&bars[SB_F0 + i], 1);
            mbar_init(&bars[SB_E0 + i], 1 + kStWorkers);
            mbar_init(&bars[SB_TF0 + i], kStTables);
            mbar_init(&bars[SB_TE0 + i], kStWorkers);
        }
        for (int i = 0; i < kPieces; ++i) {
            mbar_init(&bars[SB_WF0 + i], 4);
            mbar_init(&bars[SB_WE0 + i], 1);
        }
        mbar_init(&bars[SB_DONE], 1);
        mbar_init(&bars[SB_READ], kStWorkers);
        mbar_init(&bars[SB_END], 1);
        *abort_flag = p.timeout_test;
        fence_barrier_init();
    }
    if (warp == 2) tmem_alloc(tslot, 512);
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tslot;
    const Waiter wt{bars, abort_flag, p.status};
    auto chunk_of = [&](int j) { return nch - 1 - j; };    // from the end
    auto len_of = [&](int j) { return min(L, seg.len - chunk_of(j) * L); };
    auto stage_full = [&](int j) { return wt(SB_F0 + j % 3, (uint32_t)((j / 3) & 1)); };
    bool ok = !(p.timeout_test && warp == 1);

    if (warp == 0) {
        int issued = 0;
        for (int j = 0; j < nch; ++j) {
            const int s = j % 3;
            if (j >= 3) ok = wt(SB_E0 + s, (uint32_t)((j / 3 - 1) & 1));
            if (!ok) break;
            if (lane == 0) {
                uint8_t *st = sm + s * Cfg::STAGE;
                uint64_t *full = &bars[SB_F0 + s];
                const int t = (int)(seg.t0 + (int64_t)chunk_of(j) * L);
                const int gb = head / (p.HV / p.HK) * DK;
                mbar_arrive_expect_tx(full, Cfg::STAGE);
                tma_load_2d(st, &tm_b, full, gb, t);
                tma_load_2d(st + 16384, &tm_b, full, gb + 64, t);
#pragma unroll
                for (int q = 0; q < VT / 64; ++q)
                    tma_load_2d(st + 32768 + q * 16384, &tm_x, full, head * DV + 64 * q, t);
            }
            issued = j + 1;
            __syncwarp();
        }
        // no load stays in flight behind this CTA, whatever the other roles do
        for (int j = issued > 3 ? issued - 3 : 0; j < issued; ++j) wt.drain(SB_F0 + j % 3, (uint32_t)((j / 3) & 1));
    } else if (warp == 1) {
        const uint32_t id = idesc_bf16(128, DK, false, true);
        const bool issuer = elect_one();
        int r = 0, ph = 0;           // ring slot of the next piece and its phase
        for (int j = 0; j < nch && ok; ++j) {
            const bool fresh = j % kFlush == 0;
            if (fresh && j > 0) ok = wt(SB_READ, (uint32_t)((j / kFlush - 1) & 1));
            ok = ok && stage_full(j);
            const uint64_t b0 = sdesc_sw128(sb + (j % 3) * Cfg::STAGE, 16384, 1024);
            // (unrolled: the tensor cores hold only a few products ahead of the one that runs)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                ok = ok && wt(SB_WF0 + r, (uint32_t)ph);
                if (!ok) break;
                tc_fence_after();
                if (issuer) {
                    const uint32_t a = tmem + TS_A + r * TS_PIECE;
                    const uint32_t add = !fresh || q > 0;
                    mma_bf16_ts(tmem + TS_D, a, desc_add(b0, q * 4096), id, add);
                    mma_bf16_ts(tmem + TS_DS, a + 16, desc_add(b0, q * 4096), id, add);
                    mma_bf16_ts(tmem + TS_DS, a + 32, desc_add(b0, q * 4096), id, 1);
                    mma_bf16_ts(tmem + TS_D, a + 8, desc_add(b0, q * 4096 + 2048), id, 1);
                    mma_bf16_ts(tmem + TS_DS, a + 24, desc_add(b0, q * 4096 + 2048), id, 1);
                    mma_bf16_ts(tmem + TS_DS, a + 40, desc_add(b0, q * 4096 + 2048), id, 1);
                    mma_commit(&bars[SB_WE0 + r]);
                    if (q == 3) {
                        mma_commit(&bars[SB_E0 + j % 3]);
                        if (j % kFlush == kFlush - 1 || j == nch - 1) mma_commit(&bars[SB_DONE]);
                    }
                }
                __syncwarp();
                if (++r == kPieces) {
                    r = 0;
                    ph ^= 1;
                }
            }
        }
        // every product issued here has completed before tensor memory is released
        if (elect_one()) mma_commit(&bars[SB_END]);
        __syncwarp();
        wt.drain(SB_END, 0);
    } else if (warp < kStWork0) {
        // a 32-token block of every chunk each: the weights to the block's end, and its decay
        const int q = warp - kStTable0;
        HeadTab ht[NH];
#pragma unroll
        for (int e = 0; e < NH; ++e) ht[e] = {p.a[head + e] * kLog2e, p.dt_bias ? p.dt_bias[head + e] : 0.f};
        const float *dtp = p.dt + seg.t0 * p.HV + head;
        auto load_dt = [&](int j, int e) {
            const int t = chunk_of(j) * L + 32 * q + lane;
            return t >= 0 && t < seg.len ? __ldg(dtp + (int64_t)t * p.HV + e) : 0.f;
        };
        float ahead[NH][2];     // dt of the next two chunks
#pragma unroll
        for (int e = 0; e < NH; ++e) {
            ahead[e][0] = load_dt(0, e);
            ahead[e][1] = load_dt(1, e);
        }
#pragma unroll 1
        for (int j = 0; j < nch; ++j) {
            const int s = j % 3;
            if (j >= 3 && !wt(SB_TE0 + s, (uint32_t)((j / 3 - 1) & 1))) break;
            const bool in = chunk_of(j) * L + 32 * q + lane < seg.len;
#pragma unroll
            for (int e = 0; e < NH; ++e) {
                float delta, g, pre, suf;
                token_step(ahead[e][0], ht[e], in, p.soft, delta, g);
                ahead[e][0] = ahead[e][1];
                ahead[e][1] = load_dt(j + 2, e);
                const float sum = block_sums(g, lane, pre, suf);
                reinterpret_cast<float *>(sm + Cfg::O_TAB + (s * NH + e) * 512)[32 * q + lane] = delta * ex2(suf);
                if (lane == 0) reinterpret_cast<float *>(sm + Cfg::O_SUM + (s * NH + e) * 16)[q] = sum;
            }
            warp_arrive(&bars[SB_TF0 + s]);
        }
    } else if (warp >= kStWork0) {
        // lanes (value columns) 32 quad .. + 31; block th of every chunk is a piece, formed by
        // four warps; and columns 32 th .. + 31 of the sums
        const int quad = warp & 3, th = (warp - kStWork0) >> 2;
        const bool mine = 32 * quad < VT;                       // (a tile of 64 fills half of the lanes)
        const int e = NH == 2 ? quad >> 1 : 0;
        // this lane's row of the 8x8 blocks: token (lane & 7) + 8 of blocks 2, 3; columns + 8 of blocks 1, 3
        const int trow = 32 * th + (lane & 7) + 8 * (lane >> 4), vblk = (lane >> 3) & 1;
        const int tok = 32 * th + 2 * (lane & 3);               // this lane's tokens: + 8 b + {0, 1}
        float run = 0.f, acc[32];      // log2 decays behind the chunk; the sums
#pragma unroll
        for (int i = 0; i < 32; ++i) acc[i] = 0.f;
        for (int j = 0; j < nch && ok; ++j) {
            const int s = j % 3, len = len_of(j);
            ok = stage_full(j) && wt(SB_TF0 + s, (uint32_t)((j / 3) & 1));
            if (!ok) break;
            const uint32_t stage = sb + s * Cfg::STAGE;
            const float *tab = reinterpret_cast<const float *>(sm + Cfg::O_TAB + (s * NH + e) * 512);
            const float4 sum = *reinterpret_cast<const float4 *>(sm + Cfg::O_SUM + (s * NH + e) * 16);
            float after = run;         // ... and behind this block
            if (th < 3) after += sum.w;
            if (th < 2) after += sum.z;
            if (th < 1) after += sum.y;
            run += (sum.x + sum.y) + (sum.z + sum.w);
            const float far = ex2(after);
            const int pc = 4 * j + th, r = pc % kPieces;
            if (pc >= kPieces) ok = wt(SB_WE0 + r, (uint32_t)((pc / kPieces - 1) & 1));
            if (!ok) break;
            if (mine) {
#pragma unroll 1
                for (int b = 0; b < 2; ++b) {
                    float2 w2[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        w2[i] = mulp(*reinterpret_cast<const float2 *>(tab + tok + 16 * b + 8 * i), make_float2(far, far));
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        const int col = 32 * quad + 16 * g + 8 * vblk;
                        uint32_t x[4], hi[4], mid[4], lo[4];
                        ldsm_x4_t(stage + 32768 + (col >> 6) * 16384 + sw128_chunk(trow + 16 * b, (col & 63) >> 3), x);
                        if (len < L) {   // rows behind the sequence may hold anything
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const int t = tok + 16 * b + 8 * (i >> 1);
                                if (t >= len) x[i] = 0u;
                                if (t + 1 >= len) x[i] &= 0xffffu;
                            }
                        }
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            float2 f = mulp(unpack2(x[i]), w2[i >> 1]);
                            hi[i] = take_high(f);
                            mid[i] = take_high(f);
                            lo[i] = high_pair(f);
                        }
                        const uint32_t ta = tmem + ((uint32_t)(32 * quad + 16 * g) << 16) + TS_A + r * TS_PIECE + 8 * b;
                        tmem_st_16x128b_x2(ta, hi);
                        tmem_st_16x128b_x2(ta + 16, mid);
                        tmem_st_16x128b_x2(ta + 32, lo);
                    }
                }
                tmem_wait_st();
            }
            if (len < L) {
                // rows of b behind the sequence: a NaN there must not meet the zeros (each block's
                // by its four warps)
                for (int v = 32 * quad + lane; v < 32 * 16; v += 128) {
                    const int row = 32 * th + (v >> 4), ch = v & 15;
                    if (row >= len) sts128(stage + (ch >> 3) * 16384 + row * 128 + (ch & 7) * 16, 0, 0, 0, 0);
                }
                fence_proxy_async_smem();
            }
            tc_fence_before();
            warp_arrive(&bars[SB_WF0 + r]);
            warp_arrive(&bars[SB_E0 + s]);
            warp_arrive(&bars[SB_TE0 + s]);
            if (j % kFlush == kFlush - 1 || j == nch - 1) {
                ok = wt(SB_DONE, (uint32_t)((j / kFlush) & 1));
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    float hi[8], small[8];
                    tmem_ld8(tmem_addr(tmem, warp, TS_D + 32 * th + 8 * g), hi);
                    tmem_ld8(tmem_addr(tmem, warp, TS_DS + 32 * th + 8 * g), small);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 8; ++i) acc[8 * g + i] += hi[i] + small[i];
                }
                tc_fence_before();
                warp_arrive(&bars[SB_READ]);
            }
        }
        if (ok && mine) {
            const int row = 32 * quad + lane;
            float4 *dst = reinterpret_cast<float4 *>(
                p.seg_state + (((size_t)slot * p.HV + head + row / DV) * DV + row % DV) * DK + 32 * th);
#pragma unroll
            for (int u = 0; u < 8; ++u) dst[u] = make_float4(acc[4 * u], acc[4 * u + 1], acc[4 * u + 2], acc[4 * u + 3]);
        }
        // (quadrant 0 has the first head, quadrant 2 the second)
        if (ok && th == 0 && lane == 0 && (quad == 0 || (NH == 2 && quad == 2)))
            p.seg_decay[(size_t)slot * p.HV + head + e] = ex2(run);
    }
    __syncthreads();
    if (warp == 2) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// -------------------------------------------------------------------- the scan
template <int VT, int NH>
struct ScanCfg {
    static constexpr uint32_t XT = VT * 256;
    static constexpr uint32_t PIECE = VT * 64;               // w x of 32 tokens, bf16
    static constexpr int NS = 3;
    static constexpr uint32_t O_C = 0, O_B = 32768, O_X = O_B + 65536;
    static constexpr uint32_t O_S = O_X + 2 * XT;            // S as bf16: 128 rows (k) x VT
    static constexpr uint32_t O_W = O_S + XT;
    static constexpr int NT = 3;                             // table buffers
    static constexpr uint32_t O_TAB = O_W + NS * PIECE;      // [NT][NH] x HeadTable
    static constexpr uint32_t O_BAR = O_TAB + NT * NH * 1536;
    static constexpr uint32_t BYTES = O_BAR + 768 + 1024;
};
static_assert(ScanCfg<128, 2>::BYTES <= 232448, "shared memory");
constexpr int kScMask = 4, kScState = 8, kScWeight = 12, kScOut = 16, kScThreads = 20 * 32;
enum ScBar { B_CF, B_CE, B_BF0, B_BF1, B_BE0, B_BE1, B_XF0, B_XF1, B_XE0, B_XE1, B_TF0, B_TE0 = B_TF0 + 3,
             B_CB = B_TE0 + 3, B_P, B_S, B_UD, B_WF0, B_WE0 = B_WF0 + 3, B_Y = B_WE0 + 3, B_YE, B_CL, B_DONE, B_COUNT };
static_assert(8 * B_COUNT + 8 <= 384, "barriers");
// One head's factors of a chunk: per token the running sum of log2 decays in its
// 32-token block, delta times the decays behind it in the block, and `diag`; per block
// the sum of its log2 decays and the decays behind the block.
// A block whose decays multiply to no less than 2^-100 (kMild) has delta e^(-running sum)
// in `diag`: its diagonal tile then needs no exponential per element.  Others have delta.
constexpr float kMild = -100.f;
struct HeadTable {
    float run[L], tail[L], diag[L];
};
struct BlockTable {
    float sum[4], behind[4], all;   // (all: the decays of the whole chunk)
};
constexpr uint32_t T_CB = 0, T_Y1 = 128, T_Y2 = 256, T_S = 384;

template <int VT, int NH>
__global__ void __launch_bounds__(kScThreads, 1)
scan_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_b,
            const __grid_constant__ CUtensorMap tm_c, const __grid_constant__ CUtensorMap tm_y, const TcParams p) {
    using Cfg = ScanCfg<VT, NH>;
    constexpr int DV = VT / NH;
    extern __shared__ uint8_t raw[];
    uint8_t *sm = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
    const uint32_t sb = smem_u32(sm);
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + Cfg::O_BAR);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(sm + Cfg::O_BAR + 8 * B_COUNT);
    uint32_t *tslot = reinterpret_cast<uint32_t *>(sm + Cfg::O_BAR + 8 * B_COUNT + 4);
    BlockTable *blocks = reinterpret_cast<BlockTable *>(sm + Cfg::O_BAR + 384);   // [NT][NH]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tiles = p.HV / NH;
    int slot = blockIdx.x / tiles;
    const int head = (blockIdx.x - slot * tiles) * NH;
    if (blockIdx.x == 0 && threadIdx.x == 0 && !p.chained) *p.status = 0u;
    const Seg seg = find_seg(p.map, slot);
    if (!seg.ok || seg.len <= 0) {
        // The grid is done when its CTAs are, and what follows it in the stream then starts:
        // where no segment has a token (a packed batch of empty sequences) these CTAs are all
        // there are, and the kernels that still write hT and read the table have to be done too.
        if (p.chained) wait_for_previous();
        return;
    }
    const int nch = (seg.len + L - 1) / L, last = nch - 1;
    const int tail = seg.len - last * L;      // tokens of the last chunk
    if (threadIdx.x == 0) {
        mbar_init(&bars[B_CF], 1);
        mbar_init(&bars[B_CE], 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars[B_BF0 + i], 1);
            mbar_init(&bars[B_BE0 + i], 1);
            mbar_init(&bars[B_XF0 + i], 1);
            mbar_init(&bars[B_XE0 + i], 8);
        }
        for (int i = 0; i < Cfg::NT; ++i) {
            mbar_init(&bars[B_TF0 + i], 1);
            mbar_init(&bars[B_TE0 + i], 16);
        }
        mbar_init(&bars[B_CB], 1);
        mbar_init(&bars[B_P], 4);
        mbar_init(&bars[B_S], 4);
        mbar_init(&bars[B_UD], 1);
        for (int i = 0; i < 3; ++i) {
            mbar_init(&bars[B_WF0 + i], 4);
            mbar_init(&bars[B_WE0 + i], 1);
        }
        mbar_init(&bars[B_Y], 1);
        mbar_init(&bars[B_YE], 4);
        mbar_init(&bars[B_CL], 4);
        mbar_init(&bars[B_DONE], 1);
        *abort_flag = p.timeout_test;
        fence_barrier_init();
    }
    if (warp == 3) tmem_alloc(tslot, 512);
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tslot;
    const Waiter wt{bars, abort_flag, p.status};
    auto par2 = [](int c) { return (uint32_t)((c >> 1) & 1); };          // phase of use c >> 1 (two buffers)
    auto par2_before = [](int c) { return (uint32_t)(((c >> 1) - 1) & 1); };
    auto table = [&](int c, int e) { return reinterpret_cast<HeadTable *>(sm + Cfg::O_TAB + ((c % 3) * NH + e) * 1536); };
    auto block = [&](int c, int e) { return blocks + (c % 3) * NH + e; };
    auto table_full = [&](int c) { return wt(B_TF0 + c % 3, (uint32_t)((c / 3) & 1)); };
    bool ok = !(p.timeout_test && warp == 1);

    if (warp == 0) {
        // ------------------------------------------------ loads
        int nb = 0, nx = 0, nc = 0;
        for (int c = 0; c < nch; ++c) {
            const int s = c & 1, t = (int)(seg.t0 + (int64_t)c * L);
            const int gb = head / (p.HV / p.HK) * DK;
            // the tiles' slots come free late: what they take next is in L2 by then
            if (lane == 0 && c + 2 < nch) {
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    tma_prefetch_l2_2d(&tm_b, gb + 64 * q, t + 2 * L);
                    tma_prefetch_l2_2d(&tm_c, gb + 64 * q, t + 2 * L);
                }
#pragma unroll
                for (int q = 0; q < VT / 64; ++q) tma_prefetch_l2_2d(&tm_x, head * DV + 64 * q, t + 2 * L);
            }
            __syncwarp();
            if (c >= 2) ok = wt(B_BE0 + s, par2_before(c));
            if (!ok) break;
            if (lane == 0) {
                mbar_arrive_expect_tx(&bars[B_BF0 + s], 32768);
                tma_load_2d(sm + Cfg::O_B + s * 32768, &tm_b, &bars[B_BF0 + s], gb, t);
                tma_load_2d(sm + Cfg::O_B + s * 32768 + 16384, &tm_b, &bars[B_BF0 + s], gb + 64, t);
            }
            nb = c + 1;
            // (c before x: the one C tile's load is what the next scores wait for)
            if (c >= 1) ok = wt(B_CE, (uint32_t)((c - 1) & 1));
            if (!ok) break;
            if (lane == 0) {
                mbar_arrive_expect_tx(&bars[B_CF], 32768);
                tma_load_2d(sm + Cfg::O_C, &tm_c, &bars[B_CF], gb, t);
                tma_load_2d(sm + Cfg::O_C + 16384, &tm_c, &bars[B_CF], gb + 64, t);
            }
            nc = c + 1;
            if (c >= 2) ok = wt(B_XE0 + s, par2_before(c));
            if (!ok) break;
            if (lane == 0) {
                mbar_arrive_expect_tx(&bars[B_XF0 + s], Cfg::XT);
#pragma unroll
                for (int q = 0; q < VT / 64; ++q)
                    tma_load_2d(sm + Cfg::O_X + s * Cfg::XT + q * 16384, &tm_x, &bars[B_XF0 + s], head * DV + 64 * q, t);
            }
            nx = c + 1;
            __syncwarp();
        }
        // no load stays in flight behind this CTA, whatever the other roles do
        for (int c = nb > 2 ? nb - 2 : 0; c < nb; ++c) wt.drain(B_BF0 + (c & 1), par2(c));
        for (int c = nx > 2 ? nx - 2 : 0; c < nx; ++c) wt.drain(B_XF0 + (c & 1), par2(c));
        if (nc > 0) wt.drain(B_CF, (uint32_t)((nc - 1) & 1));
    } else if (warp == 1) {
        // ------------------------------------------------ MMAs
        const uint32_t id_cb = idesc_bf16(128, 128, false, false);
        const uint32_t id_cs = idesc_bf16(128, VT, false, true);
        const uint32_t id_px = idesc_bf16(128, DV, false, true);
        const uint32_t id_up = idesc_bf16(128, VT, true, true);
        const uint64_t cd = sdesc_sw128(sb + Cfg::O_C, 16, 1024);
        const uint64_t sd = sdesc_sw128(sb + Cfg::O_S, 16384, 1024);
        auto scores = [&](int c) {   // C B^T of chunk c
            ok = ok && wt(B_CF, (uint32_t)(c & 1)) && wt(B_BF0 + (c & 1), par2(c));
            if (c == last && tail < L) ok = ok && wt(B_CL, 0);
            if (!ok) return;
            tc_fence_after();
            const uint64_t bd = sdesc_sw128(sb + Cfg::O_B + (c & 1) * 32768, 16, 1024);
            if (elect_one()) {
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const uint32_t off = (k >> 2) * 16384 + (k & 3) * 32;
                    mma_bf16(tmem + T_CB, desc_add(cd, off), desc_add(bd, off), id_cb, k > 0);
                }
                mma_commit(&bars[B_CB]);
            }
            __syncwarp();
        };
        scores(0);
        for (int c = 0; c < nch && ok; ++c) {
            const uint32_t btile = sb + Cfg::O_B + (c & 1) * 32768, xtile = sb + Cfg::O_X + (c & 1) * Cfg::XT;
            ok = wt(B_S, (uint32_t)(c & 1));
            if (!ok) break;
            tc_fence_after();
            // S^T += B^T (w x); between its pieces, when the outputs of the chunk before have
            // been read, C S^T (it frees the one C tile for the next chunk's load)
            const uint64_t ad = sdesc_sw128(btile, 16384, 1024);
#pragma unroll 1
            for (int q = 0; q < 4 && ok; ++q) {
                if (q == 2) {
                    if (c > 0) ok = wt(B_YE, (uint32_t)((c - 1) & 1));
                    if (!ok) break;
                    tc_fence_after();
                    if (elect_one()) {
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            mma_bf16(tmem + T_Y1, desc_add(cd, (k >> 2) * 16384 + (k & 3) * 32), desc_add(sd, k * 2048),
                                     id_cs, k > 0);
                        mma_commit(&bars[B_CE]);
                    }
                    __syncwarp();
                }
                if (c == last) continue;
                const int pc = 4 * c + q, r = pc % 3;
                ok = wt(B_WF0 + r, (uint32_t)((pc / 3) & 1));
                if (!ok) break;
                tc_fence_after();
                const uint64_t wd = sdesc_sw128(sb + Cfg::O_W + r * Cfg::PIECE, 4096, 1024);
                if (elect_one()) {
                    mma_bf16(tmem + T_S, desc_add(ad, q * 4096), wd, id_up, 1);
                    mma_bf16(tmem + T_S, desc_add(ad, q * 4096 + 2048), desc_add(wd, 2048), id_up, 1);
                    mma_commit(&bars[B_WE0 + r]);
                    if (q == 3) mma_commit(&bars[B_UD]);
                }
                __syncwarp();
            }
            ok = ok && wt(B_P, (uint32_t)(c & 1)) && wt(B_XF0 + (c & 1), par2(c));
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {       // P X
#pragma unroll
                for (int e = 0; e < NH; ++e) {
                    const uint64_t xd = sdesc_sw128(xtile + e * 16384, 16384, 1024);
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        mma_bf16_ts(tmem + T_Y2 + DV * e, tmem + T_CB + 32 * (k >> 1) + 8 * (k & 1) + 16 * e,
                                    desc_add(xd, k * 2048), id_px, k > 0);
                }
                mma_commit(&bars[B_Y]);
                mma_commit(&bars[B_BE0 + (c & 1)]);
            }
            __syncwarp();
            if (c < last) scores(c + 1);
        }
        if (elect_one()) mma_commit(&bars[B_DONE]);
        __syncwarp();
        wt.drain(B_DONE, 0);
    } else if (warp == 2 || warp == 3) {
        // ------------------------------------------------ tables (every other chunk each)
        HeadTab ht[NH];
#pragma unroll
        for (int e = 0; e < NH; ++e) ht[e] = {p.a[head + e] * kLog2e, p.dt_bias ? p.dt_bias[head + e] : 0.f};
        const float *dtp = p.dt + seg.t0 * p.HV + head;
        auto load_dt = [&](int c, int q, int e) {
            const int t = c * L + 32 * q + lane;
            return t < seg.len ? __ldg(dtp + (int64_t)t * p.HV + e) : 0.f;
        };
        // four blocks of dt on their way, the one used next last
        const int first = warp - 2;
        float ahead[NH][4];
#pragma unroll
        for (int e = 0; e < NH; ++e)
#pragma unroll
            for (int q = 0; q < 4; ++q) ahead[e][q] = load_dt(first, q, e);
        for (int c = first; c < nch && ok; c += 2) {
            if (c >= 3) ok = wt(B_TE0 + c % 3, (uint32_t)((c / 3 - 1) & 1));
            if (!ok) break;
            float behind[NH];
#pragma unroll
            for (int e = 0; e < NH; ++e) behind[e] = 0.f;
#pragma unroll 1
            for (int q = 3; q >= 0; --q) {
                const bool in = c * L + 32 * q + lane < seg.len;
#pragma unroll
                for (int e = 0; e < NH; ++e) {
                    float delta, g, pre, suf;
                    token_step(ahead[e][3], ht[e], in, p.soft, delta, g);
                    ahead[e][3] = ahead[e][2];
                    ahead[e][2] = ahead[e][1];
                    ahead[e][1] = ahead[e][0];
                    ahead[e][0] = load_dt(c + 2, q, e);
                    const float sum = block_sums(g, lane, pre, suf);
                    HeadTable *tab = table(c, e);
                    tab->run[32 * q + lane] = pre;
                    tab->tail[32 * q + lane] = delta * ex2(suf);
                    tab->diag[32 * q + lane] = sum >= kMild ? delta * ex2(-pre) : delta;
                    if (lane == 0) {
                        block(c, e)->sum[q] = sum;
                        block(c, e)->behind[q] = ex2(behind[e]);
                    }
                    behind[e] += sum;
                    if (q == 0 && lane == 0) block(c, e)->all = ex2(behind[e]);
                }
            }
            warp_arrive(&bars[B_TF0 + c % 3]);
        }
    } else if (warp >= kScMask && warp < kScState) {
        // ------------------------------------------------ mask: C B^T -> P (rows i = tokens)
        const int w = warp - kScMask, i = 32 * w + lane;
        for (int c = 0; c < nch && ok; ++c) {
            ok = table_full(c) && wt(B_CB, (uint32_t)(c & 1));
            if (!ok) break;
            tc_fence_after();
#pragma unroll 1
            for (int q = 0; q < 4; ++q) {
                const uint32_t ta = tmem_addr(tmem, warp, T_CB + 32 * q);
                uint32_t out[16];
                if (q > w) {
#pragma unroll
                    for (int u = 0; u < 16; ++u) out[u] = 0u;
#pragma unroll
                    for (int e = 0; e < NH; ++e) tmem_st16w(ta + 16 * e, out);
                    continue;
                }
                float v[32];
                tmem_ld32r(ta, v);
#pragma unroll 1
                for (int e = 0; e < NH; ++e) {
                    const HeadTable *t = table(c, e);
                    const float pi = t->run[i];
                    const bool mild = block(c, e)->sum[q] >= kMild;
                    if (q < w || mild) {
                        // decays of the tokens behind block q, up to i (on the diagonal: from
                        // the block's start)
                        const BlockTable *b = block(c, e);
                        float s = pi;
                        if (q < 1 && w > 1) s += b->sum[1];
                        if (q < 2 && w > 2 && q < w) s += b->sum[2];
                        const float rf = ex2(s);
                        const float2 rf2 = make_float2(rf, rf);
                        const float4 *cf = reinterpret_cast<const float4 *>((q < w ? t->tail : t->diag) + 32 * q);
#pragma unroll
                        for (int u = 0; u < 8; ++u) {
                            const float4 f = cf[u];
                            const float2 p0 = mulp(mulp(make_float2(f.x, f.y), rf2), make_float2(v[4 * u], v[4 * u + 1]));
                            const float2 p1 = mulp(mulp(make_float2(f.z, f.w), rf2), make_float2(v[4 * u + 2], v[4 * u + 3]));
                            out[2 * u] = pack_bf16x2(p0.x, p0.y);
                            out[2 * u + 1] = pack_bf16x2(p1.x, p1.y);
                        }
                        if (q == w) {
                            // tokens behind i: the pairs with both, or the second, behind it
#pragma unroll
                            for (int u = 0; u < 16; ++u) {
                                if (2 * u > lane) out[u] = 0u;
                                if (2 * u == lane) out[u] &= 0xffffu;
                            }
                        }
                    } else {
                        // the sums from j + 1 to i one after the other, from j = i down (a running
                        // sum of thousands would leave their differences 12 bits)
                        const float4 *dj = reinterpret_cast<const float4 *>(t->diag + 32 * q);
                        const float ah = __ldg(p.a + head + e) * kLog2e;
                        float sum = 0.f;
#pragma unroll
                        for (int u = 7; u >= 0; --u) {
                            const float4 d4 = dj[u];
                            const float ds[4] = {d4.x, d4.y, d4.z, d4.w};
                            float f[4];
#pragma unroll
                            for (int b = 3; b >= 0; --b) {
                                const bool in = 4 * u + b <= lane;
                                f[b] = in ? v[4 * u + b] * (ds[b] * ex2(sum)) : 0.f;
                                sum += in ? log_decay(ds[b], ah) : 0.f;
                            }
                            out[2 * u] = pack_bf16x2(f[0], f[1]);
                            out[2 * u + 1] = pack_bf16x2(f[2], f[3]);
                        }
                    }
                    tmem_st16w(ta + 16 * e, out);
                }
            }
            tmem_wait_st();
            tc_fence_before();
            warp_arrive(&bars[B_P]);
            warp_arrive(&bars[B_TE0 + c % 3]);
        }
    } else if (warp >= kScState && warp < kScWeight) {
        // ------------------------------------------------ state (lanes k)
        const int k = 32 * (warp - kScState) + lane;
        // the start states are the only thing here that the kernels before this one make
        if (p.chained) wait_for_previous();
        const float *src = p.chained ? p.seg_state + ((size_t)slot * p.HV + head) * DV * DK
                           : p.h0    ? p.h0 + ((size_t)seg.n * p.HV + head) * DV * DK
                                     : nullptr;
#pragma unroll 1
        for (int col = 0; col < VT; col += 32) {
            uint32_t v[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = src ? __float_as_uint(src[(size_t)(col + i) * DK + k]) : 0u;
            tmem_st32(tmem_addr(tmem, warp, T_S + col), v);
        }
        tmem_wait_st();
        for (int c = 0; c < nch && ok; ++c) {
            if (c > 0) ok = wt(B_UD, (uint32_t)((c - 1) & 1)) && wt(B_CE, (uint32_t)((c - 1) & 1));
            ok = ok && table_full(c);
            if (!ok) break;
            tc_fence_after();
#pragma unroll 1
            for (int g = 0; g < VT / 32; ++g) {
                const uint32_t ta = tmem_addr(tmem, warp, T_S + 32 * g);
                float v[32];
                tmem_ld32r(ta, v);
                const uint32_t dst = sb + Cfg::O_S + (g >> 1) * 16384;
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    sts128(dst + sw128_chunk(k, 4 * (g & 1) + u), pack_bf16x2(v[8 * u], v[8 * u + 1]),
                           pack_bf16x2(v[8 * u + 2], v[8 * u + 3]), pack_bf16x2(v[8 * u + 4], v[8 * u + 5]),
                           pack_bf16x2(v[8 * u + 6], v[8 * u + 7]));
                if (c < last) {
                    const float s = block(c, (32 * g) / DV)->all;
                    const float2 s2 = make_float2(s, s);
                    uint32_t o[32];
#pragma unroll
                    for (int u = 0; u < 16; ++u) {
                        const float2 f = mulp(make_float2(v[2 * u], v[2 * u + 1]), s2);
                        o[2 * u] = __float_as_uint(f.x);
                        o[2 * u + 1] = __float_as_uint(f.y);
                    }
                    tmem_st32(ta, o);
                }
            }
            tmem_wait_st();
            fence_proxy_async_smem();
            tc_fence_before();
            warp_arrive(&bars[B_S]);
            warp_arrive(&bars[B_TE0 + c % 3]);
        }
    } else if (warp >= kScWeight && warp < kScOut) {
        // ------------------------------------------------ w x, 32 tokens a piece
        const int tid = threadIdx.x - kScWeight * 32, row = tid >> 3, pc8 = tid & 7;
        for (int c = 0; c < last && ok; ++c) {
            ok = wt(B_XF0 + (c & 1), par2(c)) && table_full(c);
            const uint32_t xtile = sb + Cfg::O_X + (c & 1) * Cfg::XT;
#pragma unroll 1
            for (int q = 0; q < 4 && ok; ++q) {
                const int pc = 4 * c + q, r = pc % 3;
                if (pc >= 3) ok = wt(B_WE0 + r, (uint32_t)((pc / 3 - 1) & 1));
                if (!ok) break;
                const uint32_t src = xtile + (32 * q + row) * 128 + pc8 * 16;
                const uint32_t dst = sb + Cfg::O_W + r * Cfg::PIECE + row * 128 + pc8 * 16;
#pragma unroll
                for (int v = 0; v < VT / 64; ++v) {
                    const float *tab = table(c, NH == 2 ? v : 0)->tail + 32 * q + row;
                    const float behind = block(c, NH == 2 ? v : 0)->behind[q];
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const uint4 u = lds128(src + v * 16384 + half * 2048);
                        const float w = tab[16 * half] * behind;
                        sts128(dst + v * 4096 + half * 2048, weighted(u.x, w), weighted(u.y, w), weighted(u.z, w),
                               weighted(u.w, w));
                    }
                }
                fence_proxy_async_smem();
                warp_arrive(&bars[B_WF0 + r]);
            }
            if (ok) {
                warp_arrive(&bars[B_XE0 + (c & 1)]);
                warp_arrive(&bars[B_TE0 + c % 3]);
            }
        }
        if (tail < L && ok) {
            // rows behind the sequence are another's (or none): a NaN there must not
            // meet P's zeros
            ok = wt(B_XF0 + (last & 1), par2(last)) && wt(B_BF0 + (last & 1), par2(last));
            if (ok) {
                const uint32_t xtile = sb + Cfg::O_X + (last & 1) * Cfg::XT, btile = sb + Cfg::O_B + (last & 1) * 32768;
                for (int r = tail + row; r < L; r += 16) {
#pragma unroll
                    for (int v = 0; v < VT / 64; ++v) sts128(xtile + v * 16384 + r * 128 + pc8 * 16, 0, 0, 0, 0);
                    sts128(btile + r * 128 + pc8 * 16, 0, 0, 0, 0);
                    sts128(btile + 16384 + r * 128 + pc8 * 16, 0, 0, 0, 0);
                }
                fence_proxy_async_smem();
                warp_arrive(&bars[B_CL]);
            }
        }
    } else if (warp >= kScOut) {
        // ------------------------------------------------ y (rows i = tokens)
        const int quad = warp & 3, i = 32 * quad + lane;
        float dh[NH];
#pragma unroll
        for (int e = 0; e < NH; ++e) dh[e] = p.d ? p.d[head + e] : 0.f;
        __nv_bfloat16 *yr = p.y + ((seg.t0 + i) * p.HV + head) * DV;
        for (int c = 0; c < nch && ok; ++c) {
            ok = table_full(c) && wt(B_XF0 + (c & 1), par2(c));
            if (!ok) break;
            float ga[NH];
#pragma unroll
            for (int e = 0; e < NH; ++e) {
                float s = table(c, e)->run[i];
#pragma unroll
                for (int m = 0; m < 3; ++m)
                    if (m < quad) s += block(c, e)->sum[m];
                ga[e] = ex2(s);
            }
            warp_arrive(&bars[B_TE0 + c % 3]);
            ok = wt(B_Y, (uint32_t)(c & 1));
            if (!ok) break;
            tc_fence_after();
            const bool whole = c < last || tail == L;
            const uint32_t xtile = sb + Cfg::O_X + (c & 1) * Cfg::XT;
#pragma unroll 1
            for (int g = 0; g < VT / 16; ++g) {
                const int col = 16 * g;
                const float gs = NH == 2 && col >= DV ? ga[NH - 1] : ga[0], ds = NH == 2 && col >= DV ? dh[NH - 1] : dh[0];
                const float2 ga2 = make_float2(gs, gs), de2 = make_float2(ds, ds);
                float v1[16], v2[16];
                tmem_ld16(tmem_addr(tmem, warp, T_Y1 + col), v1);
                tmem_ld16(tmem_addr(tmem, warp, T_Y2 + col), v2);
                const uint32_t xa = xtile + (col >> 6) * 16384;
                const int ch = (col & 63) >> 3;
                const uint4 xu = lds128(xa + sw128_chunk(i, ch)), xv = lds128(xa + sw128_chunk(i, ch + 1));
                const uint32_t xw[8] = {xu.x, xu.y, xu.z, xu.w, xv.x, xv.y, xv.z, xv.w};
                tmem_wait_ld();
                uint32_t o[8];
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    float2 f = fma2(ga2, make_float2(v1[2 * u], v1[2 * u + 1]), make_float2(v2[2 * u], v2[2 * u + 1]));
                    f = fma2(de2, unpack2(xw[u]), f);
                    o[u] = pack_bf16x2(f.x, f.y);
                }
                if (whole) {
                    // y takes x's place in the tile (the weights and P X are done with it)
                    sts128(xa + sw128_chunk(i, ch), o[0], o[1], o[2], o[3]);
                    sts128(xa + sw128_chunk(i, ch + 1), o[4], o[5], o[6], o[7]);
                } else if (i < tail) {
                    uint4 *dst = reinterpret_cast<uint4 *>(yr + 16 * g);
                    dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
                    dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
                }
            }
            tc_fence_before();
            warp_arrive(&bars[B_YE]);
            if (whole) {
                // this warp's 32 rows, by the copy engine
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
#pragma unroll
                    for (int q = 0; q < VT / 64; ++q)
                        tma_store_2d(&tm_y, xtile + q * 16384 + quad * 4096, head * DV + 64 * q,
                                     (int)(seg.t0 + (int64_t)c * L) + 32 * quad);
                    bulk_commit_group();
                    bulk_wait_group_read0();
                }
            }
            warp_arrive(&bars[B_XE0 + (c & 1)]);
            yr += (size_t)L * p.HV * DV;
        }
    }
    __syncthreads();
    if (warp == 3) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

int sm_count() {
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)
        return 148;
    return n;
}

int heads_per_tile(const SsmArgs &a) { return a.dv == 64 && (a.HV / a.HK) % 2 == 0 ? 2 : 1; }

struct TcCut {
    int seg_len, nseg;
    int64_t bound;
    size_t table, first, order, decay, state, total;
};

// Segment length in chunks: the fewest waves of CTAs over the SMs times the chunks of
// a wave, a segment counting 2 chunks more for its start and end states.  That number of
// segments goes up and down with T; the workspace has room for what any call of as many
// sequences and tokens may take, so the cuts are held to kCutWaves waves of CTAs beyond one
// segment a sequence.  (Of 4000 sizes up to 256K tokens 1.3% would take more to gain 2% of
// the chunks; with half as many waves 7% would.  8 waves are 78 MB of states.)
constexpr int kCutWaves = 8;
TcCut cut_tc(const SsmArgs &a) {
    TcCut c{};
    const bool packed = a.cu_seqlens != nullptr;
    const int64_t chunks = (a.T + L - 1) / L > 0 ? (a.T + L - 1) / L : 1, seqs = packed ? 1 : a.N;
    const int64_t tiles = a.HV / heads_per_tile(a), sms = sm_count();
    const int64_t more = kCutWaves * sms / tiles;     // segments beyond one a sequence
    int64_t best = 0, best_cost = 0;
    for (int64_t n = 1; n <= 64 && n <= chunks; ++n) {
        const int64_t len = (chunks + n - 1) / n, segs = (chunks + len - 1) / len;
        if ((segs - 1) * seqs > more) continue;
        const int64_t waves = (segs * seqs * tiles + sms - 1) / sms;
        const int64_t cost = waves * (len + 2);
        if (best == 0 || cost < best_cost) {
            best = len;
            best_cost = cost;
        }
    }
    c.seg_len = (int)(best * L);
    c.nseg = (int)((chunks + best - 1) / best);
    // (a sequence of l > 0 tokens has 1 + (l - 1) / seg_len segments)
    c.bound = packed ? a.N + c.nseg - 1 : (int64_t)a.N * c.nseg;
    const int64_t slots = a.N + min(more, (chunks - 1) * seqs);
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
    off += (size_t)slots * a.HV * a.dv * DK * sizeof(float);
    c.total = off;
    return c;
}

template <int VT, int NH>
cudaError_t launch_tiles(const SsmArgs &a, cudaStream_t stream) {
    const TcCut cut = cut_tc(a);
    const int64_t grid = cut.bound * (a.HV / NH);
    if (grid > 0x7fffffff || (int64_t)a.N * a.HV > 0x7fffffff) return cudaErrorInvalidValue;
    const bool packed = a.cu_seqlens != nullptr;
    uint8_t *ws = static_cast<uint8_t *>(a.workspace);
    const bool cuts = packed ? a.T > cut.seg_len : cut.nseg > 1;
    const bool states = cuts || a.hT != nullptr;
    // the first kernel clears the status word; with no tokens and no states to return there is none
    if (!states && a.T == 0) return cudaMemsetAsync(ws, 0, sizeof(unsigned int), stream);
    cudaError_t err = cudaSuccess;
    TcParams p{a.dt, a.a, a.d, a.dt_bias, a.h0, a.HK, a.HV, a.softplus, 
               static_cast<__nv_bfloat16 *>(a.y),
               reinterpret_cast<float *>(ws + cut.state), reinterpret_cast<float *>(ws + cut.decay),
               reinterpret_cast<unsigned int *>(ws), states, a.hT != nullptr,
               a.timeout_test,
               SegMap{nullptr, nullptr, a.N, cut.nseg, a.T, cut.seg_len}};
    if (packed) {
        p.map.table = reinterpret_cast<int4 *>(ws + cut.table);
        p.map.first = reinterpret_cast<int *>(ws + cut.first);
        int *order = cut.bound <= kOrdered ? reinterpret_cast<int *>(ws + cut.order) : nullptr;
        p.map.order = order;
        err = launch_plan(a.cu_seqlens, a.N, cut.seg_len, (int)cut.bound, reinterpret_cast<int4 *>(ws + cut.table),
                          reinterpret_cast<int *>(ws + cut.first), order, stream);
        if (err != cudaSuccess) return err;
    }
    const uint64_t tokens = (uint64_t)(packed ? a.T : (int64_t)a.N * a.T);
    CUtensorMap tx{}, tb{}, tcm{}, ty{};
    if (tokens > 0) {
        const uint32_t box[2] = {64, (uint32_t)L}, ybox[2] = {64, 32};
        const uint64_t dx[2] = {(uint64_t)a.HV * a.dv, tokens}, db[2] = {(uint64_t)a.HK * DK, tokens};
        const uint64_t sx[1] = {(uint64_t)a.x_row * 2}, sbb[1] = {(uint64_t)a.b_row * 2}, sc[1] = {(uint64_t)a.c_row * 2},
                       sy[1] = {(uint64_t)a.HV * a.dv * 2};
        if (!encode_bf16_map(&tx, a.x, 2, dx, sx, box) || !encode_bf16_map(&tb, a.b, 2, db, sbb, box) ||
            !encode_bf16_map(&tcm, a.c, 2, db, sc, box) || !encode_bf16_map(&ty, a.y, 2, dx, sy, ybox))
            return cudaErrorInvalidValue;
    }
    if (states) {
        constexpr uint32_t bytes = StatesCfg<VT, NH>::BYTES;
        err = cudaFuncSetAttribute(states_kernel<VT, NH>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
        if (err != cudaSuccess) return err;
        states_kernel<VT, NH><<<(unsigned)grid, kStThreads, bytes, stream>>>(tx, tb, p);
        err = launch_combine(p.seg_state, p.seg_decay, a.h0, a.hT, a.N, a.HV, a.dv * DK, p.whole, p.map, stream);
        if (err != cudaSuccess) return err;
    }
    if (tokens > 0) {
        constexpr uint32_t bytes = ScanCfg<VT, NH>::BYTES;
        err = cudaFuncSetAttribute(scan_kernel<VT, NH>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
        if (err != cudaSuccess) return err;
        if (states)
            return launch_after(scan_kernel<VT, NH>, dim3((unsigned)grid), dim3(kScThreads), bytes, stream, tx, tb, tcm, ty, p);
        scan_kernel<VT, NH><<<(unsigned)grid, kScThreads, bytes, stream>>>(tx, tb, tcm, ty, p);
    }
    return cudaGetLastError();
}

}  // namespace

bool tc_supported(const SsmArgs &a) { return a.dtype == GDN_BF16 && a.dk == DK && (a.dv == 64 || a.dv == 128); }
size_t tc_workspace_bytes(const SsmArgs &a) { return cut_tc(a).total; }
cudaError_t launch_tc(const SsmArgs &a, cudaStream_t stream) {
    if (a.dv == 128) return launch_tiles<128, 1>(a, stream);
    return heads_per_tile(a) == 2 ? launch_tiles<128, 2>(a, stream) : launch_tiles<64, 1>(a, stream);
}

}  // namespace ssm
}  // namespace gdn
