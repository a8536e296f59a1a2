// linear_walk.cuh -- the linear attention passes of linear_attn.h in 64-token
// chunks on the tensor cores (tcgen05, bf16 operands, float32 accumulators in
// TMEM).
//
// With G the sum of log decays within a chunk up to a token and A the state at
// the chunk's edge, a pass over a chunk is (t, s its tokens; forward shown)
//     out_t = a_t A x_t + sum_{s <= t} Gamma_ts (x_t . y_s) z_s,
//     A     <- gamma A + sum_s w_s z_s y_s^T,
//     a_t = e^{G_t},  Gamma_ts = e^{G_t - G_s},  w_s = e^{G_end - G_s},  gamma = e^{G_end};
// backward in time a and w change places and the mask is s >= t.  No exponent
// is positive.  Four products per chunk, all with 128 rows (the z index), so
// that everything the CUDA cores make is a tensor core operand read from TMEM,
// where thread = row, except the scores:
//     KV     = (w z)^T y          A operand from TMEM: three bf16 parts
//     inter  = A x^T              A operand from TMEM: A in bf16 (one part, or three)
//     P      = x y^T              both from shared memory as TMA left them
//     intra  = z^T (Gamma o P)^T  z from shared memory, the scores written there (one part, or three)
//
// Precision.  w z is split into three bf16 parts (8 bits each: exact), and the
// state is accumulated in float32 registers from one chunk's KV at a time, so
// the state is exact to float32 rounding.  Where only out is wanted, A and the
// scores enter their product rounded to bf16 (2^-8 relative); the passes whose
// dot products give the decays' gradient (kExact) take three parts of both,
// because that gradient is a difference of sums that nearly cancel.
//
// Work split.  The state chain runs along a sequence, so a sequence is cut into
// parts of L tokens: a first launch (kState) gives each part's own sum of KV, a
// scan over the parts their starting states, and the walk then takes all parts
// at once.  One CTA per (part, output head); the value heads that share an
// output row are taken in turn by one CTA, which adds them in float32.
//
// Roles in a CTA of 16 warps, handing over through mbarriers (every wait is
// bounded; one that gives up raises the workspace's error word):
//   warps 0-7    the state in registers (64 columns a thread), its bf16 copy,
//                and the output: the chunk's inter and intra
//   warps 8-11   w z in three parts, one z index a thread
//   warps 12-13  the scores, one token a thread
//   warp  14     TMA loads and the chunk's decays
//   warp  15     issues the products
#pragma once

#include <cuda.h>

#include "common.cuh"
#include "kernels.h"
#include "linear_attn.h"
#include "tc_util.cuh"

namespace gdn {
namespace lin {

using namespace tc;

enum Mode { kOut = 0, kExact = 1, kState = 2 };

constexpr int kD = 128;
constexpr int kC = 64;                          // tokens of a chunk
constexpr int kThreads = 512;
constexpr uint64_t kWaitLimitNs = 2000000000ull;
constexpr uint32_t kPanel = 64 * 128;           // 64 rows of 64 bf16, 128-byte swizzle
constexpr uint32_t kTile = 2 * kPanel;          // 64 rows of 128

// what a pass needs beyond LinPass
struct Walk {
    LinPass p;
    int32_t part_len;               // tokens of a part (a multiple of 64)
    int32_t n_parts;                // upper bound of the number of parts
    int32_t split;                  // sequences may have several parts: states at their joints in `joint`
    float* joint;                   // [n_parts, Hv, 128, 128]: a part's own sum (kState), its starting state (walk)
    int32_t joint_t;                // joint holds the transposed state
    float* joint_decay;             // [n_parts, Hv]
    uint32_t* err;
};

struct Part {
    int64_t t0, t1;                 // its tokens
    int32_t seq;                    // -1: there is no such part
    int32_t first, last;            // first and last of its sequence, in the pass's direction
    int32_t alone;                  // its sequence has one part
};

// The index-th part: sequence i has max(1, ceil(len / part_len)) parts.  One warp.
GDN_DEVICE Part find_part(const Walk& w, int32_t index) {
    const int lane = threadIdx.x & 31;
    Part r{0, 0, -1, 0, 0, 0};
    int64_t before = 0;
    for (int32_t i0 = 0; i0 < w.p.n_seq; i0 += 32) {
        const int32_t i = i0 + lane;
        int64_t a = 0, b = 0;
        int32_t n = 0;
        if (i < w.p.n_seq) {
            a = w.p.cu ? w.p.cu[i] : 0;
            b = w.p.cu ? w.p.cu[i + 1] : w.p.T;
            n = b > a ? (int32_t)((b - a + w.part_len - 1) / w.part_len) : 1;
        }
        int32_t upto = n;
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const int32_t x = __shfl_up_sync(0xffffffffu, upto, m);
            if (lane >= m) upto += x;
        }
        const int32_t k = (int32_t)(index - before) - (upto - n);        // the part's number in this lane's sequence
        const unsigned found = __ballot_sync(0xffffffffu, k >= 0 && k < n);
        if (found) {
            const int src = __ffs(found) - 1;
            if (lane == src) {
                r.t0 = a + (int64_t)k * w.part_len;
                r.t1 = r.t0 + w.part_len < b ? r.t0 + w.part_len : b;
                r.seq = i;
                r.first = w.p.backward ? k == n - 1 : k == 0;
                r.last = w.p.backward ? k == 0 : k == n - 1;
                r.alone = n == 1;
            }
            r.t0 = __shfl_sync(0xffffffffu, r.t0, src);
            r.t1 = __shfl_sync(0xffffffffu, r.t1, src);
            r.seq = __shfl_sync(0xffffffffu, r.seq, src);
            r.first = __shfl_sync(0xffffffffu, r.first, src);
            r.last = __shfl_sync(0xffffffffu, r.last, src);
            r.alone = __shfl_sync(0xffffffffu, r.alone, src);
            return r;
        }
        before += __shfl_sync(0xffffffffu, upto, 31);
    }
    return r;
}

template <int kMode>
struct Layout {
    static constexpr bool kOuts = kMode != kState;
    static constexpr int kParts = kMode == kExact ? 3 : 1;         // of A and of the scores
    // shared memory: stages of [x] y z [u] tiles, the scores, decays per stage, barriers
    static constexpr uint32_t kX = 0;
    static constexpr uint32_t kY = kOuts ? kTile : 0;
    static constexpr uint32_t kZ = kY + kTile;
    static constexpr uint32_t kU = kZ + kTile;
    static constexpr uint32_t kStage = kU + (kMode == kExact ? kTile : 0);
    static constexpr int kStages = kMode == kExact ? 3 : kMode == kOut ? 4 : 6;
    static constexpr uint32_t kScores = kStages * kStage;
    static constexpr uint32_t kGates = kScores + (kOuts ? kParts * kPanel : 0);
    // a stage's decays: a[64], w[64], exponent high and low [64] each, gamma, tokens
    static constexpr uint32_t kGateBytes = (4 * 64 + 4) * 4;
    static constexpr uint32_t kDots = kGates + kStages * kGateBytes;       // [8 warps][32] partial dot products
    static constexpr uint32_t kBars = kDots + (kMode == kExact ? 8 * 32 * 4 : 0);
    // barriers
    static constexpr int bFull = 0, bEmpty = bFull + kStages, bPFull = bEmpty + kStages, bPReady = bPFull + 1,
                         bAReady = bPReady + 1, bKvFull = bAReady + 1, bKvFree = bKvFull + 1, bOFull = bKvFree + 1,
                         bOFree = bOFull + 1, bWFull = bOFree + 1, bWFree = bWFull + 2, bZeroed = bWFree + 2,
                         bDots = bZeroed + 1, bDrain = bDots + 2, kBarCount = bDrain + 1;
    static constexpr uint32_t kMisc = kBars + ((kBarCount * 8 + 15) / 16) * 16;    // TMEM base, abort flag, part
    static constexpr uint32_t kSmem = kMisc + 64;
    static constexpr uint32_t kAlloc = kSmem + 1024;
    static_assert(kAlloc <= 232448, "a CTA's shared memory");
    // TMEM columns.  kExact: intra takes the scores' columns once they have been read.
    static constexpr uint32_t tKv = 0, tInter = 128, tP = 192, tIntra = kMode == kExact ? 192 : 256,
                              tA = kMode == kExact ? 256 : 320, tW = kMode == kExact ? 448 : 384;
    // w z is handed over in slots of this many tokens, two slots
    static constexpr int kSlot = kMode == kExact ? 16 : 32;
    static constexpr int kSlots = kC / kSlot;
    static constexpr uint32_t kSlotCols = 3 * kSlot / 2;
};
static_assert(Layout<kExact>::tW + 2 * Layout<kExact>::kSlotCols <= 512 && Layout<kOut>::tW + 2 * Layout<kOut>::kSlotCols <= 512,
              "TMEM columns");

// x = hi + mid + lo in bf16 for a pair of values: 8 bits each, cut, so that the remainders are exact
GDN_DEVICE void split3(float x0, float x1, uint32_t& hi, uint32_t& mid, uint32_t& lo) {
    const uint32_t b0 = __float_as_uint(x0), b1 = __float_as_uint(x1);
    const float r0 = x0 - __uint_as_float(b0 & 0xffff0000u), r1 = x1 - __uint_as_float(b1 & 0xffff0000u);
    const uint32_t m0 = __float_as_uint(r0), m1 = __float_as_uint(r1);
    hi = __byte_perm(b0, b1, 0x7632);
    mid = __byte_perm(m0, m1, 0x7632);
    lo = pack_bf16x2(r0 - __uint_as_float(m0 & 0xffff0000u), r1 - __uint_as_float(m1 & 0xffff0000u));
}

// ex2.approx keeps 2^-22 relative; exponents here are <= 0
GDN_DEVICE float exp2_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// everything a role needs
struct Ctx {
    const Walk& w;
    uint8_t* sm;
    uint32_t base;                  // its shared-space address
    uint32_t tmem;
    volatile int* abort;
    Part part;
    int32_t chunks;                 // of the part
    int32_t head;                   // output head (kState: value head)
    int32_t reps;                   // value heads to take in turn
    int32_t head0;                  // the first of them

    GDN_DEVICE uint32_t bar(uint32_t bars, int i) const { return base + bars + i * 8; }
    GDN_DEVICE bool wait(uint32_t bars, int i, uint32_t parity) const {
        return mbar_wait(bar(bars, i), parity & 1u, abort, kWaitLimitNs);
    }
    // first token of the n-th chunk in the pass's direction
    GDN_DEVICE int64_t chunk_start(int32_t n) const {
        return part.t0 + (int64_t)(w.p.backward ? chunks - 1 - n : n) * kC;
    }
};

// ---- warp 14: loads and decays ------------------------------------------------------------------------
template <int kMode>
GDN_DEVICE void load_role(const Ctx& c, const CUtensorMap* mx, const CUtensorMap* my, const CUtensorMap* mz,
                          const CUtensorMap* mu) {
    using L = Layout<kMode>;
    const int lane = threadIdx.x & 31;
    const LinPass& p = c.w.p;
    const int32_t total = c.reps * c.chunks;
    int32_t issued = 0;
    for (int32_t it = 0; it < total; ++it) {
        const int st = it % L::kStages;
        const int32_t n = it % c.chunks, h = c.head0 + it / c.chunks;
        if (it >= L::kStages && !c.wait(L::kBars, L::bEmpty + st, it / L::kStages - 1)) break;
        const int64_t t = c.chunk_start(n);
        const int valid = (int)min((int64_t)kC, c.part.t1 - t);
        const uint32_t full = c.bar(L::kBars, L::bFull + st);
        if (lane == 0) {
            const uint32_t s = c.base + st * L::kStage;
            mbar_arrive_expect_tx(full, L::kStage);
            for (int k = 0; k < 2; ++k) {
                if (L::kOuts) tma_load_2d(s + L::kX + k * kPanel, mx, h / p.x.rep * kD + k * 64, (int32_t)t, full);
                tma_load_2d(s + L::kY + k * kPanel, my, h / p.y.rep * kD + k * 64, (int32_t)t, full);
                tma_load_2d(s + L::kZ + k * kPanel, mz, h / p.z.rep * kD + k * 64, (int32_t)t, full);
                if (kMode == kExact) tma_load_2d(s + L::kU + k * kPanel, mu, h / p.u.rep * kD + k * 64, (int32_t)t, full);
            }
        }
        issued = it + 1;
        // the sums of log decays (base 2) in 64 bits: two tokens a lane
        const int i0 = 2 * lane, i1 = i0 + 1;
        float g0 = i0 < valid ? p.g[(t + i0) * p.ldg + h] : 0.f;
        float g1 = i1 < valid ? p.g[(t + i1) * p.ldg + h] : 0.f;
        g0 = g0 < kLinMinLogDecay ? kLinMinLogDecay : g0;
        g1 = g1 < kLinMinLogDecay ? kLinMinLogDecay : g1;
        const double kLog2e = 1.4426950408889634;
        const double d0 = (double)g0 * kLog2e, d1 = (double)g1 * kLog2e;
        double upto = d0 + d1;
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const double x = __shfl_up_sync(0xffffffffu, upto, m);
            if (lane >= m) upto += x;
        }
        const double all = __shfl_sync(0xffffffffu, upto, 31);
        const double G0 = upto - d1, G1 = upto;
        float* gate = reinterpret_cast<float*>(c.sm + L::kGates + st * L::kGateBytes);
        const float e0 = exp2f((float)G0), e1 = exp2f((float)G1);                // from the chunk's start
        const float f0 = exp2f((float)(all - G0)), f1 = exp2f((float)(all - G1));    // to its end
        const bool bw = p.backward != 0;
        const float ws = bw ? p.scale : 1.f;
        reinterpret_cast<float2*>(gate)[lane] = make_float2(bw ? f0 : e0, bw ? f1 : e1);
        reinterpret_cast<float2*>(gate + 64)[lane] = make_float2(i0 < valid ? ws * (bw ? e0 : f0) : 0.f,
                                                                 i1 < valid ? ws * (bw ? e1 : f1) : 0.f);
        // the exponent of Gamma_ts is E_t - E_s; as high (a multiple of 2^-10, so that differences of the
        // high parts are exact: |E| < 64 * 151) and low part
        const double E0 = bw ? -G0 : G0, E1 = bw ? -G1 : G1;
        const double h0 = rint(E0 * 1024.0) * (1.0 / 1024.0), h1 = rint(E1 * 1024.0) * (1.0 / 1024.0);
        reinterpret_cast<float2*>(gate + 128)[lane] = make_float2((float)h0, (float)h1);
        reinterpret_cast<float2*>(gate + 192)[lane] = make_float2((float)(E0 - h0), (float)(E1 - h1));
        if (lane == 0) {
            gate[256] = exp2f((float)all);
            reinterpret_cast<int32_t*>(gate)[257] = valid;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(full);
    }
    // loads still in flight land before the CTA may exit
    volatile int no_abort = 0;
    for (int32_t it = issued > L::kStages ? issued - L::kStages : 0; it < issued; ++it)
        mbar_wait(c.bar(L::kBars, L::bFull + it % L::kStages), (it / L::kStages) & 1, &no_abort, kWaitLimitNs);
}

// ---- warp 15: products ---------------------------------------------------------------------------------
template <int kMode>
GDN_DEVICE void mma_role(const Ctx& c) {
    using L = Layout<kMode>;
    if ((threadIdx.x & 31) != 0) return;
    constexpr uint32_t idKv = idesc_bf16(128, 128, false, true);
    constexpr uint32_t idKK = idesc_bf16(128, 64, false, false);
    constexpr uint32_t idPv = idesc_bf16(128, 64, true, false);
    const int32_t total = c.reps * c.chunks;
    const uint64_t dScores = sdesc_sw128(c.base + L::kScores, 16, 1024);
    auto k_major = [&](int st, uint32_t tile) { return sdesc_sw128(c.base + st * L::kStage + tile, 16, 1024); };
    auto mn_major = [&](int st, uint32_t tile) { return sdesc_sw128(c.base + st * L::kStage + tile, kPanel, 1024); };
    auto k_step = [](int kk) { return (uint64_t)(((kk >> 2) * kPanel + (kk & 3) * 32) >> 4); };
    auto commit = [&](int b) { mma_commit(c.bar(L::kBars, b)); };
    // P = x y^T of chunk it
    auto scores = [&](int32_t it) {
        const int st = it % L::kStages;
        const uint64_t dx = k_major(st, L::kX), dy = k_major(st, L::kY);
        for (int kk = 0; kk < 8; ++kk) mma_bf16(c.tmem + L::tP, dx + k_step(kk), dy + k_step(kk), idKK, kk > 0);
        commit(L::bPFull);
    };
    bool ok = true;
    if (kMode == kOut && total > 0) {
        ok = c.wait(L::kBars, L::bFull, 0);
        tc_fence_after();
        if (ok) scores(0);
    }
    for (int32_t it = 0; ok && it < total; ++it) {
        const int st = it % L::kStages;
        if (!c.wait(L::kBars, L::bFull + st, it / L::kStages)) break;
        // KV = (w z)^T y, slot by slot; its accumulator has been read for the chunk before
        const uint64_t dy = mn_major(st, L::kY);
        for (int s = 0; ok && s < L::kSlots; ++s) {
            const int32_t i = it * L::kSlots + s;
            ok = c.wait(L::kBars, L::bWFull + (i & 1), i >> 1);
            if (ok && s == 0 && it > 0) ok = c.wait(L::kBars, L::bKvFree, it - 1);
            if (!ok) break;
            tc_fence_after();
            const uint32_t a = c.tmem + L::tW + (i & 1) * L::kSlotCols;
            // smallest part first: the accumulator's rounding is then that of the largest part alone
            for (int part = 2; part >= 0; --part)
                for (int kk = 0; kk < L::kSlot / 16; ++kk)
                    mma_bf16_ta(c.tmem + L::tKv, a + part * (L::kSlot / 2) + kk * 8,
                                dy + (s * (L::kSlot / 16) + kk) * 128, idKv, s > 0 || part < 2 || kk > 0);
            commit(L::bWFree + (i & 1));
        }
        if (!ok) break;
        commit(L::bKvFull);
        if (kMode == kState) {
            commit(L::bEmpty + st);
            continue;
        }
        // inter and intra have been read for the chunk before
        if (it > 0 && !c.wait(L::kBars, L::bOFree, it - 1)) break;
        if (kMode == kExact) {
            tc_fence_after();
            scores(it);
        }
        if (!c.wait(L::kBars, L::bAReady, it)) break;
        tc_fence_after();
        const uint64_t dx = k_major(st, L::kX);
        for (int part = L::kParts - 1; part >= 0; --part)
            for (int kk = 0; kk < 8; ++kk)
                mma_bf16_ta(c.tmem + L::tInter, c.tmem + L::tA + part * 64 + kk * 8, dx + k_step(kk), idKK,
                            part < L::kParts - 1 || kk > 0);
        if (!c.wait(L::kBars, L::bPReady, it)) break;
        if (kMode == kOut && it + 1 < total) {
            if (!c.wait(L::kBars, L::bFull + (it + 1) % L::kStages, (it + 1) / L::kStages)) break;
            tc_fence_after();
            scores(it + 1);
        }
        tc_fence_after();
        const uint64_t dz = mn_major(st, L::kZ);
        for (int part = L::kParts - 1; part >= 0; --part)
            for (int kk = 0; kk < 4; ++kk)
                mma_bf16(c.tmem + L::tIntra, dz + kk * 128, dScores + part * (kPanel >> 4) + kk * 2, idPv,
                         part < L::kParts - 1 || kk > 0);
        commit(L::bOFull);
        commit(L::bEmpty + st);
    }
    // products still in flight end before TMEM is freed
    volatile int no_abort = 0;
    commit(L::bDrain);
    mbar_wait(c.bar(L::kBars, L::bDrain), 0, &no_abort, kWaitLimitNs);
}

// ---- warps 8-11: w z in three parts ---------------------------------------------------------------------
template <int kMode>
GDN_DEVICE void weight_role(const Ctx& c) {
    using L = Layout<kMode>;
    const int lane = threadIdx.x & 31, quad = (threadIdx.x >> 5) & 3;
    const int z = quad * 32 + lane;                            // this thread's z index
    const uint32_t lanes = (uint32_t)(quad * 32) << 16;
    const int32_t total = c.reps * c.chunks;
    uint32_t zeroed = 0;
    // element (s, z) of a tile: panel z >> 6, row s, 16-byte piece (z & 63) >> 3 swizzled by s & 7
    uint32_t at[8];
#pragma unroll
    for (int r = 0; r < 8; ++r)
        at[r] = (z >> 6) * kPanel + sw128_off(r, (z & 63) >> 3) + (z & 7) * 2;
    for (int32_t it = 0; it < total; ++it) {
        const int st = it % L::kStages;
        if (!c.wait(L::kBars, L::bFull + st, it / L::kStages)) return;
        uint8_t* stage = c.sm + st * L::kStage;
        const float* gate = reinterpret_cast<const float*>(c.sm + L::kGates + st * L::kGateBytes);
        const int valid = reinterpret_cast<const int32_t*>(gate)[257];
        if (valid < kC) {
            // rows of y and z behind the part's last token belong to others and may hold anything: their
            // weights and scores are 0, and 0 times a NaN is not
            for (int i = threadIdx.x & 127; i < (kC - valid) * 32; i += 128) {
                const int row = valid + (i >> 5), piece = i & 31;
                uint8_t* tile = stage + (piece & 16 ? L::kZ : L::kY) + ((piece >> 3) & 1) * kPanel;
                *reinterpret_cast<uint4*>(tile + row * 128 + (piece & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(c.bar(L::kBars, L::bZeroed));
            if (!c.wait(L::kBars, L::bZeroed, zeroed++)) return;
        }
        const uint8_t* tile = stage + L::kZ;
        for (int s = 0; s < L::kSlots; ++s) {
            const int32_t i = it * L::kSlots + s;
            if (i >= 2 && !c.wait(L::kBars, L::bWFree + (i & 1), (i >> 1) - 1)) return;
            tc_fence_after();
            const uint32_t dst = c.tmem + lanes + L::tW + (i & 1) * L::kSlotCols;
#pragma unroll
            for (int kk = 0; kk < L::kSlot / 16; ++kk) {
                uint32_t part[3][8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int t = s * L::kSlot + kk * 16 + 2 * j;
                    const float2 w = *reinterpret_cast<const float2*>(gate + 64 + t);
                    const float z0 = bf16_to_f32(*reinterpret_cast<const uint16_t*>(tile + at[(2 * j) & 7] + (t >> 3) * 1024));
                    const float z1 = bf16_to_f32(*reinterpret_cast<const uint16_t*>(tile + at[(2 * j + 1) & 7] + (t >> 3) * 1024));
                    split3(w.x * z0, w.y * z1, part[0][j], part[1][j], part[2][j]);
                }
#pragma unroll
                for (int k = 0; k < 3; ++k) tmem_st8u(dst + k * (L::kSlot / 2) + kk * 8, part[k]);
            }
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(c.bar(L::kBars, L::bWFull + (i & 1)));
        }
    }
}

// ---- warps 12-13: scores ----------------------------------------------------------------------------------
template <int kMode>
GDN_DEVICE void score_role(const Ctx& c) {
    using L = Layout<kMode>;
    const int lane = threadIdx.x & 31, quad = (threadIdx.x >> 5) & 3;      // 0 or 1
    const int t = quad * 32 + lane;
    const uint32_t lanes = (uint32_t)(quad * 32) << 16;
    const int32_t total = c.reps * c.chunks;
    const bool bw = c.w.p.backward != 0;
    for (int32_t it = 0; it < total; ++it) {
        const int st = it % L::kStages;
        if (!c.wait(L::kBars, L::bFull + st, it / L::kStages)) return;
        const float* gate = reinterpret_cast<const float*>(c.sm + L::kGates + st * L::kGateBytes);
        const int valid = reinterpret_cast<const int32_t*>(gate)[257];
        const float eh = gate[128 + t], el = gate[192 + t];
        if (!c.wait(L::kBars, L::bPFull, it)) return;
        tc_fence_after();
        // the scores of the chunk before have been used
        if (it > 0 && !c.wait(L::kBars, L::bOFull, it - 1)) return;
        uint8_t* row = c.sm + L::kScores;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            // the half above (backward: below) the diagonal of this warp's rows is empty
            const bool empty = bw ? (quad == 1 && half == 0) : (quad == 0 && half == 1);
            if (empty) {
#pragma unroll
                for (int k = 0; k < L::kParts; ++k)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        *reinterpret_cast<uint4*>(row + k * kPanel + sw128_off(t, half * 4 + j)) = make_uint4(0u, 0u, 0u, 0u);
                continue;
            }
            float p[32];
            tmem_ld32w(c.tmem + lanes + L::tP + half * 32, p);
#pragma unroll
            for (int j = 0; j < 32; j += 4) {
                const int s = half * 32 + j;
                const float4 sh = *reinterpret_cast<const float4*>(gate + 128 + s);
                float d[4] = {eh - sh.x, eh - sh.y, eh - sh.z, eh - sh.w};
                const float4 sl = *reinterpret_cast<const float4*>(gate + 192 + s);
                d[0] += el - sl.x; d[1] += el - sl.y; d[2] += el - sl.z; d[3] += el - sl.w;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const bool keep = bw ? (s + e >= t && s + e < valid) : (s + e <= t);
                    p[j + e] = keep ? p[j + e] * exp2_fast(d[e]) : 0.f;
                }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t v[L::kParts][4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float p0 = p[j * 8 + 2 * e], p1 = p[j * 8 + 2 * e + 1];
                    if (kMode == kExact) split3(p0, p1, v[0][e], v[L::kParts > 1 ? 1 : 0][e], v[L::kParts > 2 ? 2 : 0][e]);
                    else v[0][e] = pack_bf16x2(p0, p1);
                }
#pragma unroll
                for (int k = 0; k < L::kParts; ++k)
                    *reinterpret_cast<uint4*>(row + k * kPanel + sw128_off(t, half * 4 + j)) =
                        make_uint4(v[k][0], v[k][1], v[k][2], v[k][3]);
            }
        }
        fence_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(c.bar(L::kBars, L::bPReady));
    }
}

// ---- warps 0-7: state and output ----------------------------------------------------------------------------
// Thread (quad, half, lane): row z = 32 quad + lane of the state, columns 64 half .. + 64; of the output, z index
// z and the chunk's tokens 32 half .. + 32.
template <int kMode>
GDN_DEVICE void put_state(const Ctx& c, uint32_t lanes, int half, const float* S) {
    using L = Layout<kMode>;
    const uint32_t dst = c.tmem + lanes + L::tA + half * 32;
#pragma unroll
    for (int j = 0; j < 64; j += 16) {
        uint32_t v[3][8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if (kMode == kExact) split3(S[j + 2 * e], S[j + 2 * e + 1], v[0][e], v[1][e], v[2][e]);
            else v[0][e] = pack_bf16x2(S[j + 2 * e], S[j + 2 * e + 1]);
        }
#pragma unroll
        for (int k = 0; k < L::kParts; ++k) tmem_st8u(dst + k * 64 + j / 2, v[k]);
    }
    tmem_st_wait();
    tc_fence_before();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(c.bar(L::kBars, L::bAReady));
}

GDN_DEVICE void load_state(float* S, const float* src, bool transposed, int z, int half) {
    if (!src) {
#pragma unroll
        for (int j = 0; j < 64; ++j) S[j] = 0.f;
    } else if (transposed) {
#pragma unroll
        for (int j = 0; j < 64; ++j) S[j] = src[(half * 64 + j) * kD + z];
    } else {
#pragma unroll
        for (int j = 0; j < 64; j += 4) {
            const float4 v = *reinterpret_cast<const float4*>(src + z * kD + half * 64 + j);
            S[j] = v.x; S[j + 1] = v.y; S[j + 2] = v.z; S[j + 3] = v.w;
        }
    }
}

GDN_DEVICE void store_state(const float* S, float* dst, bool transposed, int z, int half) {
    if (transposed) {
#pragma unroll
        for (int j = 0; j < 64; ++j) dst[(half * 64 + j) * kD + z] = S[j];
    } else {
#pragma unroll
        for (int j = 0; j < 64; j += 4)
            *reinterpret_cast<float4*>(dst + z * kD + half * 64 + j) = make_float4(S[j], S[j + 1], S[j + 2], S[j + 3]);
    }
}

template <int kMode>
GDN_DEVICE void state_role(const Ctx& c) {
    using L = Layout<kMode>;
    const LinPass& p = c.w.p;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, quad = warp & 3, half = warp >> 2;
    const int z = quad * 32 + lane;
    const uint32_t lanes = (uint32_t)(quad * 32) << 16;
    const int heads = p.Hv / p.out_rep;
    const float fa = p.backward ? 1.f : p.scale, fp = p.scale;
    float S[64];
    int32_t it = 0;
    for (int r = 0; r < c.reps; ++r) {
        const int h = c.head0 + r;
        const int64_t own = ((int64_t)c.part.seq * p.Hv + h) * (kD * kD);
        const int64_t joint = ((int64_t)(blockIdx.x / (kMode == kState ? p.Hv : heads)) * p.Hv + h) * (kD * kD);
        if (kMode == kState) load_state(S, nullptr, false, z, half);
        else if (c.w.split && !c.part.alone) load_state(S, c.w.joint + joint, c.w.joint_t != 0, z, half);
        else load_state(S, p.init ? p.init + own : nullptr, p.state_t != 0, z, half);
        if (L::kOuts && c.chunks > 0) put_state<kMode>(c, lanes, half, S);
        for (int32_t n = 0; n < c.chunks; ++n, ++it) {
            const int st = it % L::kStages;
            if (!c.wait(L::kBars, L::bFull + st, it / L::kStages)) return;
            const float* gate = reinterpret_cast<const float*>(c.sm + L::kGates + st * L::kGateBytes);
            const float gamma = gate[256];
            if (!c.wait(L::kBars, L::bKvFull, it)) return;
            tc_fence_after();
#pragma unroll
            for (int j = 0; j < 64; j += 32) {
                float kv[32];
                tmem_ld32w(c.tmem + lanes + L::tKv + half * 64 + j, kv);
#pragma unroll
                for (int e = 0; e < 32; ++e) S[j + e] = fmaf(gamma, S[j + e], kv[e]);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(c.bar(L::kBars, L::bKvFree));
            if (kMode == kState) {
                if (lane == 0) mbar_arrive(c.bar(L::kBars, L::bEmpty + st));
                continue;
            }
            // inter has read the state's bf16 copy, and inter and intra are complete
            if (!c.wait(L::kBars, L::bOFull, it)) return;
            tc_fence_after();
            if (n + 1 < c.chunks) put_state<kMode>(c, lanes, half, S);
            const int64_t t0 = c.chunk_start(n);
            const int valid = (int)min((int64_t)kC, c.part.t1 - t0);
#pragma unroll
            for (int b = 0; b < 32; b += 16) {
                const int tb = half * 32 + b;
                float inter[16], out[16];
                tmem_ld16x2w(c.tmem + lanes + L::tInter + tb, c.tmem + lanes + L::tIntra + tb, inter, out);
#pragma unroll
                for (int e = 0; e < 16; e += 4) {
                    const float4 a = *reinterpret_cast<const float4*>(gate + tb + e);
                    out[e] = fmaf(fa * a.x, inter[e], fp * out[e]);
                    out[e + 1] = fmaf(fa * a.y, inter[e + 1], fp * out[e + 1]);
                    out[e + 2] = fmaf(fa * a.z, inter[e + 2], fp * out[e + 2]);
                    out[e + 3] = fmaf(fa * a.w, inter[e + 3], fp * out[e + 3]);
                }
                const int64_t row = ((t0 + tb) * heads + c.head) * kD + z;
                const int64_t step = (int64_t)heads * kD;
                const int rows = valid - tb;
                if (kMode == kExact) {
                    // u_t . out_t over the warp's 32 z indices: at each step lanes m apart exchange the half
                    // of their sums that the other one keeps
                    float dot[16];
                    const uint8_t* u = c.sm + st * L::kStage + L::kU + (z >> 6) * kPanel + (z & 7) * 2;
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const int t = tb + e;
                        const float uv = bf16_to_f32(*reinterpret_cast<const uint16_t*>(u + sw128_off(t, (z & 63) >> 3)));
                        dot[e] = uv * out[e];
                    }
#pragma unroll
                    for (int m = 1, hf = 8; hf >= 1; m <<= 1, hf >>= 1)
#pragma unroll
                        for (int e = 0; e < hf; ++e) {
                            const float give = (lane & m) ? dot[e] : dot[e + hf];
                            const float keep = (lane & m) ? dot[e + hf] : dot[e];
                            dot[e] = keep + __shfl_xor_sync(0xffffffffu, give, m);
                        }
                    dot[0] += __shfl_xor_sync(0xffffffffu, dot[0], 16);
                    const int e = ((lane & 1) << 3) | ((lane & 2) << 1) | ((lane & 4) >> 1) | ((lane & 8) >> 3);
                    if (lane < 16)
                        reinterpret_cast<float*>(c.sm + L::kDots)[warp * 32 + b + e] = dot[0];
                }
                if (p.out_rep > 1) {
                    float* acc = p.out_bf16 ? p.acc : static_cast<float*>(p.out);
                    if (r > 0)
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            if (e < rows) out[e] += acc[row + e * step];
                    if (r + 1 < c.reps) {
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            if (e < rows) acc[row + e * step] = out[e];
                        continue;
                    }
                }
                if (p.out_bf16) {
                    uint16_t* o = static_cast<uint16_t*>(p.out) + row;
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        if (e < rows) o[e * step] = (uint16_t)f32_to_bf16_bits(out[e]);
                } else {
                    float* o = static_cast<float*>(p.out) + row;
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        if (e < rows) o[e * step] = out[e];
                }
            }
            tc_fence_before();
            if (kMode == kExact) {
                // (the next chunk's sums are written after every warp has arrived below)
                __syncwarp();
                if (lane == 0) mbar_arrive(c.bar(L::kBars, L::bDots + half));
                if (!c.wait(L::kBars, L::bDots + half, it)) return;
                if (quad == 0 && half * 32 + lane < valid) {
                    const float* d = reinterpret_cast<const float*>(c.sm + L::kDots) + half * 128 + lane;
                    p.dots[(int64_t)h * p.T + t0 + half * 32 + lane] = (d[0] + d[32]) + (d[64] + d[96]);
                }
            }
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(c.bar(L::kBars, L::bOFree));
                mbar_arrive(c.bar(L::kBars, L::bEmpty + st));
            }
        }
        if (kMode == kState) {
            store_state(S, c.w.joint + joint, false, z, half);
        } else if (p.fin && c.part.last) {
            store_state(S, p.fin + own, p.state_t != 0, z, half);
        }
    }
}

template <int kMode>
__global__ void __launch_bounds__(kThreads, 1)
lin_walk_kernel(const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap my,
                const __grid_constant__ CUtensorMap mz, const __grid_constant__ CUtensorMap mu,
                const __grid_constant__ Walk w) {
    using L = Layout<kMode>;
    extern __shared__ uint8_t raw[];
    uint8_t* sm = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
    const uint32_t base = smem_u32(sm);
    const int warp = threadIdx.x >> 5;
    const int heads = kMode == kState ? w.p.Hv : w.p.Hv / w.p.out_rep;
    const int32_t index = (int32_t)(blockIdx.x / heads);
    const Part part = find_part(w, index);
    // kState: the last part's own sum is not needed
    if (part.seq < 0 || (kMode == kState && part.last)) return;
    volatile int* abort = reinterpret_cast<volatile int*>(sm + L::kMisc + 8);
    if (threadIdx.x == 0) {
        auto init = [&](int i, uint32_t n) { mbar_init(base + L::kBars + i * 8, n); };
        for (int s = 0; s < L::kStages; ++s) {
            init(L::bFull + s, 2);                  // the loads' bytes; the decays
            init(L::bEmpty + s, 1 + 8);             // the products; warps 0-7
        }
        init(L::bPFull, 1);
        init(L::bPReady, 2);
        init(L::bAReady, 8);
        init(L::bKvFull, 1);
        init(L::bKvFree, 8);
        init(L::bOFull, 1);
        init(L::bOFree, 8);
        for (int s = 0; s < 2; ++s) {
            init(L::bWFull + s, 4);
            init(L::bWFree + s, 1);
        }
        init(L::bZeroed, 4);
        init(L::bDots, 4);
        init(L::bDots + 1, 4);
        init(L::bDrain, 1);
        *abort = 0;
        fence_mbar_init();
    }
    if (warp == 15) tmem_alloc(base + L::kMisc, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(sm + L::kMisc);
    const int head = (int)(blockIdx.x - (unsigned)index * heads);
    const int reps = kMode == kState ? 1 : w.p.out_rep;
    const Ctx c{w, sm, base, tmem, abort, part, (int32_t)((part.t1 - part.t0 + kC - 1) / kC), head, reps, head * reps};
    if (warp < 8) {
        state_role<kMode>(c);
    } else if (warp < 12) {
        weight_role<kMode>(c);
    } else if (warp < 14) {
        if (kMode != kState) score_role<kMode>(c);
    } else if (warp == 14) {
        load_role<kMode>(c, &mx, &my, &mz, &mu);
    } else {
        mma_role<kMode>(c);
    }
    if (kMode == kState && warp == 13) {
        // the part's whole decay
        double sum = 0.0;
        for (int64_t t = part.t0 + (threadIdx.x & 31); t < part.t1; t += 32) {
            const float g = w.p.g[t * w.p.ldg + head];
            sum += g < kLinMinLogDecay ? kLinMinLogDecay : g;
        }
#pragma unroll
        for (int m = 16; m >= 1; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
        if ((threadIdx.x & 31) == 0) w.joint_decay[(int64_t)index * w.p.Hv + head] = (float)exp(sum);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (*abort && threadIdx.x == 0) *w.err = 1u;
    if (warp == 15) tmem_dealloc(tmem, 512);
}

}  // namespace lin
}  // namespace gdn
