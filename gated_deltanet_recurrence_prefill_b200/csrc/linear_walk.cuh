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
//     intra  = z^T (Gamma o P)^T  z from shared memory, the scores written there (two parts, or three)
//
// Precision.  w z is split into three bf16 parts (8 bits each: exact), and the
// state is accumulated in float32 registers from one chunk's KV at a time, so
// the state is exact to float32 rounding.  Where only out is wanted, whatever its
// type, A enters its product rounded to bf16 (2^-8 relative at most, 1.7e-3 in the
// mean, 128 independent roundings a sum) and the
// scores in two parts (2^-16): one score's rounding would be that of a whole row
// of out, and with few tokens nothing averages it (in one part, the error of a
// short call against 64 bits rose from 1.4 to 1.6 times that of out's own
// rounding).  The passes whose dot products give the decays' gradient (kExact)
// take three parts of both, because that gradient is a difference of sums that
// nearly cancel.
//
// Work split.  The state chain runs along a sequence, so a sequence is cut into
// parts of L tokens: a first launch (kState) gives each part's own sum of KV, a
// scan over the parts their starting states, and the walk then takes all parts
// at once.  One CTA per (part, output head); the value heads that share an
// output row are taken in turn by one CTA, which adds them in float32.
//
// Roles in a CTA of 28 warps, handing over through mbarriers:
//   warps 0-7    the state in registers (64 columns a thread), its bf16 copy
//   warps 8-15   the output: the chunk's inter and intra   (kState: one of them, decays)
//   warps 16-19  w z in three parts (kState: the even slots)
//   warps 20-23  the scores         (kState: w z, the odd slots)
//   warp  24     TMA loads
//   warp  25     issues KV's products
//   warp  26     issues the others   (kState: every other chunk's)
//   warp  27     the chunk's decays; it waits for every stage to come round, and for
//                the other roles to end, at most two seconds each, and makes every
//                other wait give up when that is over (the error word is raised)
// Measured (8,192 tokens, 16 / 48 heads, float32 state): kState 44 us, kOut 103 us
// (the tensor pipe 34%, HBM 29%, issue slots 57% busy), kExact 188 us (26%, 47%,
// 52%); 65,536 tokens: kOut 730 us, 3,900 cycles a chunk with all that surrounds it.
// Calls one after another: a prefill 146 us, of 65,536 tokens 1.00 ms (1.16 ms each by
// itself), a backward 680 us (720).  What bounds it is issue slots (2,000 instructions
// a chunk and scheduler) and the hand-overs between the roles, so:
//  - w z and u are read, and the output is written, as transposed 8 x 8 matrices
//    (ldmatrix / stmatrix), whose fragments are those of TMEM's 16-lane shapes; with
//    two-byte accesses the shared-memory pipe took 16 cycles each (7,300 cycles a chunk);
//  - the output leaves by TMA, and float32 pairs go through two-wide instructions;
//  - x is loaded twice, one copy below the other, so that the scores' product has
//    every row in two TMEM quadrants and four warps share them;
//  - two threads issue products: one of them alone was busy throughout (4,400 cycles).
#pragma once

#include <cuda.h>

#include "common.cuh"
#include "kernels.h"
#include "launch_chain.h"
#include "linear_attn.h"
#include "tc_util.cuh"

namespace gdn {
namespace lin {

using namespace tc;

enum Mode { kOut = 0, kExact = 1, kState = 2 };

constexpr int kD = 128;
constexpr int kC = 64;                          // tokens of a chunk
constexpr int kThreads = 896;
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
    int32_t opens;                  // the first kernel of its call: clears the error word
    // with many sequences, their parts written out beforehand (else NULL): the sequence of each part (-1: no such
    // part), the parts that are not their sequence's last, each sequence's first part
    const int32_t* part_seq;        // [n_parts]
    const int32_t* inner;           // [n_inner]
    const int32_t* seq_first;       // [n_seq + 1]
    int32_t n_inner;                // upper bound of the number of parts that are not the last
};

// Passes of one launch: the backward's two of a kind are independent of each other, and short sequences do not fill
// the GPU with one of them (a scan takes the pair too).  Kernels of their own for one pass and for two: an index into
// the parameters, where there is only one, costs the dq and dk passes 25%.
struct WalkPair {
    Walk w[2];
};
template <int kPasses>
struct Passes {
    CUtensorMap x[kPasses], y[kPasses], z[kPasses], u[kPasses], out[kPasses];
    Walk w[kPasses];
    int32_t blocks;                 // of each pass
};

struct Part {
    int64_t t0, t1;                 // its tokens
    int32_t seq;                    // -1: there is no such part
    int32_t slot;                   // its number among all parts
    int32_t first, last;            // first and last of its sequence, in the pass's direction
    int32_t alone;                  // its sequence has one part
};

// parts of a sequence: one at least
GDN_DEVICE int32_t parts_of(const Walk& w, int32_t a, int32_t b) {
    return b > a ? (int32_t)(((uint32_t)(b - a) + (uint32_t)w.part_len - 1u) / (uint32_t)w.part_len) : 1;
}

// The index-th part, or the index-th of those that are not the last of their sequence in the pass's direction.  One
// warp; without the written-out lists at most 32 sequences.
GDN_DEVICE Part find_part(const Walk& w, int32_t index, bool inner) {
    const int lane = threadIdx.x & 31;
    Part r{0, 0, -1, index, 0, 0, 0};
    const int skip = w.p.backward ? 1 : 0;      // backward in time a sequence's last part is its first one
    int32_t k = 0, n = 1, a = 0, b = 0;
    if (!w.split) {
        if (index >= w.p.n_seq || inner) return r;
        r.seq = index;
    } else if (w.part_seq) {
        if (inner) {
            r.slot = index < w.n_inner ? w.inner[index] : -1;
            if (r.slot < 0) return r;
            r.slot += skip;
        }
        r.seq = w.part_seq[r.slot];
        if (r.seq < 0) return r;
        const int32_t first = w.seq_first[r.seq];
        k = r.slot - first;
        n = w.seq_first[r.seq + 1] - first;
    } else {
        int32_t mine = 0;
        if (lane < w.p.n_seq) mine = parts_of(w, w.p.cu ? w.p.cu[lane] : 0, w.p.cu ? w.p.cu[lane + 1] : (int32_t)w.p.T);
        int32_t upto = mine;
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const int32_t x = __shfl_up_sync(0xffffffffu, upto, m);
            if (lane >= m) upto += x;
        }
        // the number in this lane's sequence (each of the sequences up to it has one part that is not inner)
        const int32_t kk = inner ? index - (upto - mine - min(lane, w.p.n_seq)) : index - (upto - mine);
        const unsigned found = __ballot_sync(0xffffffffu, kk >= 0 && kk < (inner ? mine - 1 : mine));
        if (!found) return r;
        r.seq = __ffs(found) - 1;
        k = __shfl_sync(0xffffffffu, kk, r.seq) + (inner ? skip : 0);
        n = __shfl_sync(0xffffffffu, mine, r.seq);
        r.slot = __shfl_sync(0xffffffffu, upto, r.seq) - n + k;
    }
    a = w.p.cu ? w.p.cu[r.seq] : 0;
    b = w.p.cu ? w.p.cu[r.seq + 1] : (int32_t)w.p.T;
    r.t0 = a + (int64_t)k * w.part_len;
    r.t1 = r.t0 + w.part_len < b ? r.t0 + w.part_len : b;
    r.first = w.p.backward ? k == n - 1 : k == 0;
    r.last = w.p.backward ? k == 0 : k == n - 1;
    r.alone = n == 1;
    return r;
}

// registers of the warpgroups: launched with 72 each
constexpr int kRegsState = 104, kRegsOut = 56, kRegsScores = 56, kRegsRest = 56;
static_assert(2 * kRegsState + 2 * kRegsOut + 72 + kRegsScores + kRegsRest <= 7 * 72, "the launch's registers");

template <int kMode>
struct Layout {
    static constexpr bool kOuts = kMode != kState;
    static constexpr int kParts = kMode == kExact ? 3 : 1;         // of A
    static constexpr int kScoreParts = kMode == kExact ? 3 : 2;
    // shared memory: stages of [x twice] y z [u] tiles, the scores, decays per stage, barriers
    static constexpr uint32_t kX = 0;                              // per panel: 64 rows, and the same again
    static constexpr uint32_t kY = kOuts ? 2 * kTile : 0;
    static constexpr uint32_t kZ = kY + kTile;
    static constexpr uint32_t kU = kZ + kTile;
    static constexpr uint32_t kStage = kU + (kMode == kExact ? kTile : 0);
    static constexpr int kStages = kMode == kExact ? 2 : kMode == kOut ? 3 : 6;
    // a chunk's output before it leaves, over x and y: per half of its tokens panels of 32 rows of 128 bytes
    // (64 bf16 or 32 float32), 128-byte swizzle
    static constexpr uint32_t kRows = 32 * 128, kHalf = 4 * kRows;
    static_assert(!kOuts || 2 * kHalf <= kZ, "the output's rows");
    static constexpr uint32_t kScores = kStages * kStage;
    static constexpr uint32_t kGates = kScores + (kOuts ? kScoreParts * kPanel : 0);
    // a stage's decays: a[64], w[64], exponent high and low [64] each, gamma, tokens; 4 flags: z indices 32 i .. of
    // the chunk have an infinity or NaN, each of them the first token with one in kBad[128] (int32)
    static constexpr uint32_t kFlags = (4 * 64 + 4) * 4;
    static constexpr uint32_t kGateBytes = kFlags + 16;
    static constexpr uint32_t kBad = kGates + kStages * kGateBytes;
    static constexpr uint32_t kDots = kBad + (kOuts ? kStages * 128 * 4 : 0);       // [2][8 warps][32] partial dot products
    static constexpr uint32_t kBars = kDots + (kMode == kExact ? 2 * 8 * 32 * 4 : 0);
    // the scores, and intra in their place, in one or two sets of columns; KV too
    static constexpr int kPSets = kMode == kOut ? 2 : 1, kKvSets = kMode == kState ? 2 : 1;
    // w z is handed over in slots of this many tokens
    static constexpr int kSlot = kMode == kState ? 32 : 16;
    static constexpr int kSlots = kC / kSlot;
    static constexpr int kSlotBufs = kMode == kExact ? 2 : 4;
    static constexpr uint32_t kSlotCols = 3 * kSlot / 2;
    // barriers
    static constexpr int bFull = 0, bEmpty = bFull + kStages, bPFull = bEmpty + kStages, bPReady = bPFull + 1,
                         bAReady = bPReady + 1, bKvFull = bAReady + 1, bKvFree = bKvFull + 2, bOFull = bKvFree + 2,
                         bOFree = bOFull + 1, bWFull = bOFree + 1, bWFree = bWFull + kSlotBufs, bZeroed = bWFree + kSlotBufs,
                         bRows = bZeroed + 1, bDrain = bRows + 4, bDone = bDrain + 2, bStateIn = bDone + 1,
                         bZDone = bStateIn + 1, kBarCount = bZDone + 4;
    static constexpr uint32_t kMisc = kBars + ((kBarCount * 8 + 15) / 16) * 16;    // TMEM base, abort flag, a part's decay
    static constexpr uint32_t kSmem = kMisc + 64;
    static constexpr uint32_t kAlloc = kSmem + 1024;
    static_assert(kAlloc <= 232448, "a CTA's shared memory");
    // TMEM columns.  Intra takes the scores' columns once they have been read.
    static constexpr uint32_t tKv = 0, tInter = kKvSets * 128, tP = tInter + 64, tA = tP + kPSets * 64,
                              tW = kMode == kState ? tInter : tA + kParts * 64;
    static_assert(tW + kSlotBufs * kSlotCols <= 512, "TMEM columns");
};

// pairs of float32 operations in one instruction
GDN_DEVICE float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
        "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
GDN_DEVICE float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "mul.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
GDN_DEVICE float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
GDN_DEVICE float2 sub2(float2 a, float2 b) { return fma2(b, make_float2(-1.f, -1.f), a); }

// x = hi + mid + lo in bf16 for a pair of values: 8 bits each, cut, so that the remainders are exact
GDN_DEVICE void split3(float2 x, uint32_t& hi, uint32_t& mid, uint32_t& lo) {
    const uint32_t b0 = __float_as_uint(x.x), b1 = __float_as_uint(x.y);
    const float2 r = sub2(x, make_float2(__uint_as_float(b0 & 0xffff0000u), __uint_as_float(b1 & 0xffff0000u)));
    const uint32_t m0 = __float_as_uint(r.x), m1 = __float_as_uint(r.y);
    const float2 l = sub2(r, make_float2(__uint_as_float(m0 & 0xffff0000u), __uint_as_float(m1 & 0xffff0000u)));
    hi = __byte_perm(b0, b1, 0x7632);
    mid = __byte_perm(m0, m1, 0x7632);
    lo = pack_bf16x2(l.x, l.y);
}

// x = hi + lo in bf16, the rest below 2^-16 of x
GDN_DEVICE void split2(float2 x, uint32_t& hi, uint32_t& lo) {
    const uint32_t b0 = __float_as_uint(x.x), b1 = __float_as_uint(x.y);
    const float2 r = sub2(x, make_float2(__uint_as_float(b0 & 0xffff0000u), __uint_as_float(b1 & 0xffff0000u)));
    hi = __byte_perm(b0, b1, 0x7632);
    lo = pack_bf16x2(r.x, r.y);
}

// a b + c for a pair of bf16
GDN_DEVICE uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}

// ex2.approx keeps 2^-22 relative; exponents here are <= 0
GDN_DEVICE float exp2_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// the stages in turn: index and parity of its uses
template <int kStages>
struct Ring {
    int st = 0;
    uint32_t phase = 0;
    GDN_DEVICE void next() {
        if (++st == kStages) {
            st = 0;
            phase ^= 1u;
        }
    }
};

// everything a role needs
struct Ctx {
    const Walk& w;
    uint8_t* sm;
    uint32_t base;                  // its shared-space address
    uint32_t tmem;
    volatile int* abort;
    uint32_t abort_at;              // its shared-space address
    Part part;
    int32_t chunks;                 // of the part
    int32_t head;                   // output head (kState: value head)
    int32_t reps;                   // value heads to take in turn
    int32_t head0;                  // the first of them

    GDN_DEVICE uint32_t bar(uint32_t bars, int i) const { return base + bars + i * 8; }
    GDN_DEVICE bool wait(uint32_t bars, int i, uint32_t parity) const {
        return mbar_wait_watched(bar(bars, i), parity & 1u, abort_at);
    }
    // the it-th use of a barrier, or of kSets barriers in turn
    template <int kSets>
    GDN_DEVICE bool wait_set(uint32_t bars, int i, uint32_t it) const {
        return kSets == 2 ? wait(bars, i + (int)(it & 1u), it >> 1) : wait(bars, i, it);
    }
    // first token of the n-th chunk in the pass's direction
    GDN_DEVICE int64_t chunk_start(int32_t n) const {
        return part.t0 + (int64_t)(w.p.backward ? chunks - 1 - n : n) * kC;
    }
};

GDN_DEVICE void commit_to(const Ctx& c, uint32_t bars, int i) { mma_commit(c.bar(bars, i)); }

// ---- warp 24: loads ----------------------------------------------------------------------------------
template <int kMode>
GDN_DEVICE void load_role(const Ctx& c, const CUtensorMap* mx, const CUtensorMap* my, const CUtensorMap* mz,
                          const CUtensorMap* mu) {
    using L = Layout<kMode>;
    if ((threadIdx.x & 31) != 0) return;
    const LinPass& p = c.w.p;
    Ring<L::kStages> ring;
    int32_t it = 0;
    for (int r = 0; r < c.reps; ++r) {
        const int h = c.head0 + r;
        const int32_t x0 = h / p.x.rep * kD, y0 = h / p.y.rep * kD, z0 = h / p.z.rep * kD;
        const int32_t u0 = kMode == kExact ? h / p.u.rep * kD : 0;
        int32_t t = (int32_t)c.chunk_start(0);
        const int32_t step = p.backward ? -kC : kC;
#pragma unroll 1
        for (int32_t n = 0; n < c.chunks; ++n, ++it, t += step, ring.next()) {
            if (it >= L::kStages && !c.wait(L::kBars, L::bEmpty + ring.st, ring.phase ^ 1u)) goto out;
            // the starting state comes in through the last stage
            if (kMode == kOut && it == L::kStages - 1 && !c.wait(L::kBars, L::bStateIn, 0)) goto out;
            const uint32_t full = c.bar(L::kBars, L::bFull + ring.st), s = c.base + ring.st * L::kStage;
            mbar_arrive_expect_tx(full, L::kStage);
#pragma unroll 1
            for (int k = 0; k < 2; ++k) {
                tma_load_2d(s + L::kY + k * kPanel, my, y0 + k * 64, t, full);
                if (L::kOuts) {
                    tma_load_2d(s + L::kX + k * kTile, mx, x0 + k * 64, t, full);
                    tma_load_2d(s + L::kX + k * kTile + kPanel, mx, x0 + k * 64, t, full);
                }
                tma_load_2d(s + L::kZ + k * kPanel, mz, z0 + k * 64, t, full);
                if (kMode == kExact) tma_load_2d(s + L::kU + k * kPanel, mu, u0 + k * 64, t, full);
            }
        }
    }
out:
    // loads still in flight land before the CTA may exit: the last use of each stage
    volatile int no_abort = 0;
#pragma unroll 1
    for (int k = 0; k < L::kStages && it > 0; ++k) {
        if (ring.st == 0) ring.phase ^= 1u;
        ring.st = ring.st == 0 ? L::kStages - 1 : ring.st - 1;
        --it;
        mbar_wait(c.bar(L::kBars, L::bFull + ring.st), ring.phase, &no_abort, kWaitLimitNs);
    }
}

// ---- warp 27: decays -----------------------------------------------------------------------------------
// Sums of log decays to base 2 as two integers, multiples of 2^-10 and of 2^-32 (a token's high part is below 151 *
// 2^10, its low part at most 2^21): every sum and difference in a chunk is exact, at one 32-bit addition each.
// kState: two warps take the chunks in turn (one alone, at 1,300 cycles a chunk, was the slowest role).
template <int kMode>
GDN_DEVICE void decay_role(const Ctx& c, int which, int stride) {
    using L = Layout<kMode>;
    const int lane = threadIdx.x & 31;
    const LinPass& p = c.w.p;
    const bool bw = p.backward != 0;
    const float ws = bw ? p.scale : 1.f;
    const int i0 = 2 * lane, i1 = i0 + 1;                       // this lane's tokens
    auto split = [](float g, int& hi, int& lo) {
        // exp of what is beyond these limits is 0 or inf in float32
        g = g < kLinMinLogDecay ? kLinMinLogDecay : g > -kLinMinLogDecay ? -kLinMinLogDecay : g;
        // g log2(e), the constant in two parts
        const float x = g * 1.44269502f;
        const float rest = fmaf(g, 1.44269502f, -x) + g * 1.92596303e-8f;
        hi = __float2int_rn(x * 1024.f);
        lo = __float2int_rn((fmaf((float)hi, -1.f / 1024.f, x) + rest) * 4294967296.f);
    };
    auto high = [](int x) { return (float)x * (1.f / 1024.f); };
    auto low = [](int x) { return (float)x * (1.f / 4294967296.f); };
    Ring<L::kStages> ring;
    if (which == 1) ring.next();
    int32_t it = which;
    long long whole = 0;                        // kState: the sum over this warp's chunks, multiples of 2^-32
    float whole_bad = 0.f;
    for (int r = 0; r < c.reps; ++r) {
        // this lane's log decays, fetched two chunks ahead
        const int64_t step = (int64_t)(bw ? -kC : kC) * stride;
        int64_t t = c.chunk_start(which), ahead = t;
        const float* g = p.g + c.head0 + r + (t + i0) * p.ldg;
        int32_t left = c.chunks - which;                        // not yet fetched
        auto fetch = [&](float& a, float& b) {
            a = left > 0 && ahead + i0 < c.part.t1 ? g[0] : 0.f;
            b = left > 0 && ahead + i1 < c.part.t1 ? g[p.ldg] : 0.f;
            left -= stride;
            ahead += step;
            g += step * p.ldg;
        };
        float n0, n1, m0, m1;
        fetch(n0, n1);
        fetch(m0, m1);
#pragma unroll 1
        for (int32_t n = which; n < c.chunks; n += stride, it += stride, t += step) {
            const float g0 = n0, g1 = n1;
            const int valid = (int)min((int64_t)kC, c.part.t1 - t);
            n0 = m0;
            n1 = m1;
            fetch(m0, m1);
            // a NaN reaches every sum that has its token
            const unsigned nan0 = __ballot_sync(0xffffffffu, g0 != g0), nan1 = __ballot_sync(0xffffffffu, g1 != g1);
            const unsigned earlier = (1u << lane) - 1u;
            int h0, l0, h1, l1;
            split(g0, h0, l0);
            split(g1, h1, l1);
            int H1 = h0 + h1, L1 = l0 + l1;
#pragma unroll
            for (int m = 1; m < 32; m <<= 1) {
                const int x = __shfl_up_sync(0xffffffffu, H1, m), y = __shfl_up_sync(0xffffffffu, L1, m);
                H1 += lane >= m ? x : 0;
                L1 += lane >= m ? y : 0;
            }
            const int H0 = H1 - h1, L0 = L1 - l1;
            const int allH = __shfl_sync(0xffffffffu, H1, 31), allL = __shfl_sync(0xffffffffu, L1, 31);
            const float bad = (nan0 | nan1) ? __int_as_float(0x7fc00000) : 0.f;          // added where a NaN counts
            if (kMode == kState) {
                whole += ((long long)allH << 22) + allL;
                whole_bad += bad;
            }
            // (sums up to a token: a NaN at it or before it; sums behind it: one after it)
            const float bad0 = (((nan0 | nan1) & earlier) | (nan0 & (1u << lane))) ? bad : 0.f;
            const float bad1 = (bad0 != bad0 || (nan1 & (1u << lane))) ? bad : 0.f;
            const float behind1 = ((nan0 | nan1) & ~earlier & ~(1u << lane)) ? bad : 0.f;
            const float behind0 = (nan1 & (1u << lane)) ? bad : behind1;
            const float e0 = exp2_fast(high(H0) + low(L0) + bad0), e1 = exp2_fast(high(H1) + low(L1) + bad1);
            const float f0 = exp2_fast(high(allH - H0) + low(allL - L0) + behind0);
            const float f1 = exp2_fast(high(allH - H1) + low(allL - L1) + behind1);
            // (the bound of all waits of the CTA: a stage comes round within kWaitLimitNs)
            if (it >= L::kStages &&
                !mbar_wait(c.bar(L::kBars, L::bEmpty + ring.st), ring.phase ^ 1u, c.abort, kWaitLimitNs))
                return;
            float* gate = reinterpret_cast<float*>(c.sm + L::kGates + ring.st * L::kGateBytes);
            reinterpret_cast<float2*>(gate)[lane] = make_float2(bw ? f0 : e0, bw ? f1 : e1);
            reinterpret_cast<float2*>(gate + 64)[lane] = make_float2(i0 < valid ? ws * (bw ? e0 : f0) : 0.f,
                                                                     i1 < valid ? ws * (bw ? e1 : f1) : 0.f);
            // (no NaN here: an out_t whose decays have one gets it from a_t, and the scores between tokens on the same
            // side of it stay)
            // the exponent of Gamma_ts is E_t - E_s: high parts, whose differences are exact however far strong decays have
            // taken them, and low ones
            const float sg = bw ? -1.f : 1.f;
            reinterpret_cast<float2*>(gate + 128)[lane] = make_float2(sg * high(H0), sg * high(H1));
            reinterpret_cast<float2*>(gate + 192)[lane] = make_float2(sg * low(L0), sg * low(L1));
            if (lane == 31) {
                gate[256] = e1;                                 // the whole chunk's decay
                reinterpret_cast<int32_t*>(gate)[257] = valid;
                if (L::kOuts) *reinterpret_cast<uint4*>(c.sm + L::kGates + ring.st * L::kGateBytes + L::kFlags) = make_uint4(0u, 0u, 0u, 0u);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(c.bar(L::kBars, L::bFull + ring.st));
            for (int k = 0; k < stride; ++k) ring.next();
        }
    }
    if (kMode == kState && lane == 0) {
        reinterpret_cast<long long*>(c.sm + L::kMisc + 16)[which] = whole;
        reinterpret_cast<float*>(c.sm + L::kMisc + 32)[which] = whole_bad;
    }
}

// ---- warps 25 and 26: products ---------------------------------------------------------------------------
// (Unrolled: in rolled loops an issue took up to 200 cycles, more than any of these products.)
template <int kMode>
GDN_DEVICE uint64_t k_major(const Ctx& c, int st, uint32_t tile) {
    return sdesc_sw128(c.base + st * Layout<kMode>::kStage + tile, 16, 1024);
}
template <int kMode>
GDN_DEVICE uint64_t mn_major(const Ctx& c, int st, uint32_t tile) {
    return sdesc_sw128(c.base + st * Layout<kMode>::kStage + tile, kPanel, 1024);
}

// products still in flight end before TMEM is freed
GDN_DEVICE void drain(const Ctx& c, uint32_t bar) {
    volatile int no_abort = 0;
    mma_commit(bar);
    mbar_wait(bar, 0, &no_abort, kWaitLimitNs);
}

// KV = (w z)^T y, slot by slot.  kState: two threads take the chunks in turn, one set of columns each, so that the
// tensor core has the other's products while one waits and commits.
template <int kMode>
GDN_DEVICE void kv_role(const Ctx& c, int which) {
    using L = Layout<kMode>;
    if ((threadIdx.x & 31) != 0) return;
    constexpr uint32_t idKv = idesc_bf16(128, 128, false, true);
    const int32_t total = c.reps * c.chunks;
    constexpr int kKvSets = L::kKvSets;
    Ring<L::kStages> ring;
    bool ok = true;
    if (which == 1) ring.next();
#pragma unroll 1
    for (int32_t it = which; it < total; it += kKvSets) {
        if (!c.wait(L::kBars, L::bFull + ring.st, ring.phase)) break;
        // the accumulator has been read for the chunk that used it last
        if (it >= kKvSets && !c.template wait_set<kKvSets>(L::kBars, L::bKvFree, it - kKvSets)) break;
        const int set = kKvSets == 2 ? it & 1 : 0;
        const uint64_t dy = mn_major<kMode>(c, ring.st, L::kY);
        const uint32_t d = c.tmem + L::tKv + set * 128;
#pragma unroll
        for (int s = 0; s < L::kSlots; ++s) {
            const int use = it * L::kSlots + s, buf = use % L::kSlotBufs;
            ok = c.wait(L::kBars, L::bWFull + buf, use / L::kSlotBufs);
            if (!ok) break;
            tc_fence_after();
            // smallest part first: the accumulator's rounding is then that of the largest part alone
#pragma unroll
            for (int part = 2; part >= 0; --part)
#pragma unroll
                for (int kk = 0; kk < L::kSlot / 16; ++kk)
                    mma_bf16_ta(d, c.tmem + L::tW + buf * L::kSlotCols + part * (L::kSlot / 2) + kk * 8,
                                dy + (s * (L::kSlot / 16) + kk) * 128, idKv, s > 0 || part < 2 || kk > 0);
            commit_to(c, L::kBars, L::bWFree + buf);
        }
        if (!ok) break;
        commit_to(c, L::kBars, L::bKvFull + set);
        commit_to(c, L::kBars, L::bEmpty + ring.st);
        for (int k = 0; k < kKvSets; ++k) ring.next();
    }
    drain(c, c.bar(L::kBars, L::bDrain + which));
}

// inter = A x^T, intra = z^T scores^T, and P = x y^T of the chunk after (kExact: of the chunk itself, since intra
// takes P's only columns)
template <int kMode>
GDN_DEVICE void out_products_role(const Ctx& c) {
    using L = Layout<kMode>;
    if ((threadIdx.x & 31) != 0) return;
    constexpr uint32_t idKK = idesc_bf16(128, 64, false, false);
    constexpr uint32_t idPv = idesc_bf16(128, 64, true, false);
    const int32_t total = c.reps * c.chunks;
    const uint64_t dScores = sdesc_sw128(c.base + L::kScores, 16, 1024);
    auto scores = [&](int st, uint32_t set) {
        const uint64_t dx = k_major<kMode>(c, st, L::kX), dy = k_major<kMode>(c, st, L::kY);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
            mma_bf16(c.tmem + L::tP + set, dx + (((kk >> 2) * kTile + (kk & 3) * 32) >> 4),
                     dy + (((kk >> 2) * kPanel + (kk & 3) * 32) >> 4), idKK, kk > 0);
        commit_to(c, L::kBars, L::bPFull);
    };
    Ring<L::kStages> ring;
    // kOut: the extra first turn issues chunk 0's scores
#pragma unroll 1
    for (int32_t it = kMode == kOut ? -1 : 0; it < total; ++it) {
        const uint32_t set = L::kPSets == 2 ? (it & 1) * 64 : 0;
        if (it >= 0) {
            const int st = ring.st;
            if (kMode == kExact && !c.wait(L::kBars, L::bFull + st, ring.phase)) break;
            // inter and intra have been read for the chunk before
            if (it > 0 && !c.wait(L::kBars, L::bOFree, it - 1)) break;
            if (kMode == kExact) {
                tc_fence_after();
                scores(st, 0);
            }
            if (!c.wait(L::kBars, L::bAReady, it)) break;
            tc_fence_after();
            const uint64_t dx = k_major<kMode>(c, st, L::kX);
#pragma unroll
            for (int part = L::kParts - 1; part >= 0; --part)
#pragma unroll
                for (int kk = 0; kk < 8; ++kk)
                    mma_bf16_ta(c.tmem + L::tInter, c.tmem + L::tA + part * 64 + kk * 8,
                                dx + (((kk >> 2) * kTile + (kk & 3) * 32) >> 4), idKK, part < L::kParts - 1 || kk > 0);
            // the weights' warps have looked through z (four barriers in turn: they are at most two chunks ahead, and a phase
            // passed twice would look like one to come)
            if (!c.wait(L::kBars, L::bZDone + (it & 3), it >> 2)) break;
            if (!c.wait(L::kBars, L::bPReady, it)) break;
            tc_fence_after();
            const uint64_t dz = mn_major<kMode>(c, st, L::kZ);
#pragma unroll
            for (int part = L::kScoreParts - 1; part >= 0; --part)
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    mma_bf16(c.tmem + L::tP + set, dz + kk * 128, dScores + part * (kPanel >> 4) + kk * 2, idPv,
                             part < L::kScoreParts - 1 || kk > 0);
            commit_to(c, L::kBars, L::bOFull);
            commit_to(c, L::kBars, L::bEmpty + st);
            ring.next();
        }
        if (kMode == kOut && it + 1 < total) {
            // (the other set was read for the chunk before, whose release has been waited for above)
            if (!c.wait(L::kBars, L::bFull + ring.st, ring.phase)) break;
            tc_fence_after();
            scores(ring.st, set ^ 64u);
        }
    }
    drain(c, c.bar(L::kBars, L::bDrain + 1));
}

// rows valid .. 63 of a tile, by the 128 threads of a warpgroup
GDN_DEVICE void clear_rows(uint8_t* tile, int valid) {
#pragma unroll 1
    for (int i = threadIdx.x & 127; i < (kC - valid) * 16; i += 128)
        *reinterpret_cast<uint4*>(tile + ((i >> 3) & 1) * kPanel + (valid + (i >> 4)) * 128 + (i & 7) * 16) =
            make_uint4(0u, 0u, 0u, 0u);
}

// ---- infinities and NaN in z ---------------------------------------------------------------------------------
// A token's z meets the scores of the tokens in front of it too, which are 0, and 0 times an infinity or NaN is not.
// The weights' warps, which have all of z in their hands, look for them (one bf16 product with 0 per pair: 0 unless one
// is not finite).  Where a warp finds one among its 32 z indices it leaves zeros in its place, once its weights are
// made, for intra to read, and the output's warps put NaN into those elements of out from that token on.  The search
// costs 0.8% of a long prefill and intra's wait for it 1.5%; in the scores' warps it cost 5%, in warp 27 29%, and intra
// issued without waiting, and again where something was found, 15% (more code in the roles' loops).

// `first`: of each z index the first such token in the pass's direction (past the chunk if there is none)
GDN_DEVICE void clean_z(uint8_t* tile, int32_t* first, int quad, int lane, int valid, bool bw) {
    const int z = quad * 32 + lane;
    int at = bw ? -1 : kC;
    __syncwarp();                               // every lane's rows have been read
#pragma unroll 1
    for (int t = 0; t < valid; ++t) {
        uint16_t* x = reinterpret_cast<uint16_t*>(tile + (z >> 6) * kPanel + sw128_off(t, (z & 63) >> 3)) + (z & 7);
        if ((*x & 0x7f80u) == 0x7f80u) {
            *x = 0;
            if (bw || at == kC) at = t;
        }
    }
    first[z] = at;
}

// ---- warps 16-19 (kState: 16-23): w z in three parts ------------------------------------------------------
// One warpgroup takes all slots (first = 0, stride = 1), or two take every other one.
template <int kMode>
GDN_DEVICE void weight_role(const Ctx& c, int first, int stride) {
    using L = Layout<kMode>;
    const int lane = threadIdx.x & 31, quad = (threadIdx.x >> 5) & 3;
    const uint32_t lanes = (uint32_t)(quad * 32) << 16;
    const int32_t total = c.reps * c.chunks;
    uint32_t zeroed = 0;
    Ring<L::kStages> ring;
    // This warp's z indices 32 quad .. + 32 as four 8 x 8 matrices (8 tokens each way) per ldmatrix: matrix m of
    // 16 tokens is tokens 8 (m >> 1), z indices 8 (m & 1) (+ 16 for the second half); lane l gives row l % 8 of
    // matrix l / 8.  Rows are 128 bytes, 16-byte pieces swizzled by the row.
    const int row = ((lane >> 4) << 3) + (lane & 7);            // token of 16
    const int z = quad * 32 + ((lane >> 3) & 1) * 8;
    const uint32_t at = L::kZ + (z >> 6) * kPanel + sw128_off(row, (z & 63) >> 3);
    const uint32_t at2 = L::kZ + (z >> 6) * kPanel + sw128_off(row, ((z + 16) & 63) >> 3);
#pragma unroll 1
    for (int32_t it = 0; it < total; ++it, ring.next()) {
        const int st = ring.st;
        if (!c.wait(L::kBars, L::bFull + st, ring.phase)) return;
        const float* gate = reinterpret_cast<const float*>(c.sm + L::kGates + st * L::kGateBytes);
        const int valid = reinterpret_cast<const int32_t*>(gate)[257];
        if (valid < kC) {
            // rows of y and z behind the part's last token belong to others and may hold anything: their
            // weights and scores are 0, and 0 times a NaN is not
            clear_rows(c.sm + st * L::kStage + L::kY, valid);
            clear_rows(c.sm + st * L::kStage + L::kZ, valid);
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(c.bar(L::kBars, L::bZeroed));
            if (!c.wait(L::kBars, L::bZeroed, zeroed++)) return;
        }
        const uint32_t tile = c.base + st * L::kStage;
        // 16 tokens x 16 z indices at a time, the next matrices requested before these are worked on
        uint32_t v[4], next[4], odd = 0u;
        ldmatrix_x4_trans(tile + at + first * L::kSlot * 128, next);
#pragma unroll 1
        for (int s = first; s < L::kSlots; s += stride) {
            // (a barrier's phase before its first completes at once)
            const uint32_t use = it * L::kSlots + s, buf = use % L::kSlotBufs;
            if (!c.wait(L::kBars, L::bWFree + buf, use / L::kSlotBufs + 1)) return;
            tc_fence_after();
            const uint32_t dst = c.tmem + lanes + L::tW + buf * L::kSlotCols;
#pragma unroll 1
            for (int t = s * L::kSlot; t < (s + 1) * L::kSlot; t += 16) {
                // tokens t + 8 j + 2 (lane % 4) and the next
                const float2 w0 = *reinterpret_cast<const float2*>(gate + 64 + t + 2 * (lane & 3));
                const float2 w1 = *reinterpret_cast<const float2*>(gate + 64 + t + 8 + 2 * (lane & 3));
#pragma unroll
                for (int hz = 0; hz < 2; ++hz) {
#pragma unroll
                    for (int m = 0; m < 4; ++m) {
                        v[m] = next[m];
                        if (L::kOuts) odd = fma_bf16x2(v[m], 0u, odd);
                    }
                    // (after a slot's last tokens the next slot's, which its first ones are when the stride is 1; past
                    // the chunk's end the first ones again, unused)
                    ldmatrix_x4_trans(tile + (hz ? at : at2) + ((t + 16 * hz) & (kC - 1)) * 128, next);
                    uint32_t part[3][4];
#pragma unroll
                    for (int m = 0; m < 4; ++m)
                        split3(mul2(m < 2 ? w0 : w1, bf16x2_to_f32x2(v[m])), part[0][m], part[1][m], part[2][m]);
#pragma unroll
                    for (int k = 0; k < 3; ++k)
                        tmem_st_frag8u(dst + ((uint32_t)(hz * 16) << 16) + k * (L::kSlot / 2) + (t & (L::kSlot - 1)) / 2,
                                       part[k]);
                }
            }
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(c.bar(L::kBars, L::bWFull + buf));
        }
        if (L::kOuts) {
            if (__any_sync(0xffffffffu, (odd & 0x7fff7fffu) != 0u)) {
                clean_z(c.sm + st * L::kStage + L::kZ, reinterpret_cast<int32_t*>(c.sm + L::kBad + st * 512), quad, lane, valid,
                        c.w.p.backward != 0);
                if (lane == 0) reinterpret_cast<uint32_t*>(c.sm + L::kGates + st * L::kGateBytes + L::kFlags)[quad] = 1u;
                fence_async_smem();
                __syncwarp();
            }
            if (lane == 0) mbar_arrive(c.bar(L::kBars, L::bZDone + (it & 3)));
        }
    }
}

// ---- warps 20-23: scores ----------------------------------------------------------------------------------
// TMEM lanes 64-127 repeat 0-63.  Of the 32 x 32 blocks of scores one is empty, two are cut by the diagonal: the
// rows with one block share it (16 columns a warp, and as much of the empty one to write), the others take one each.
template <int kMode>
GDN_DEVICE void score_role(const Ctx& c) {
    using L = Layout<kMode>;
    const int lane = threadIdx.x & 31, quad = (threadIdx.x >> 5) & 3;
    const int t = (quad & 1) * 32 + lane;
    const uint32_t lanes = (uint32_t)(quad * 32) << 16;
    const int32_t total = c.reps * c.chunks;
    const bool bw = c.w.p.backward != 0;
    const bool two = ((quad & 1) == 0) == bw;                   // this row block has two blocks of scores
    const int first = two ? (quad >> 1) * 32 : (bw ? 32 : 0) + (quad >> 1) * 16;
    const int empty = (bw ? 0 : 32) + (quad >> 1) * 16;
    Ring<L::kStages> ring;
#pragma unroll 1
    for (int32_t it = 0; it < total; ++it, ring.next()) {
        const int st = ring.st;
        if (!c.wait(L::kBars, L::bFull + st, ring.phase)) return;
        const float* gate = reinterpret_cast<const float*>(c.sm + L::kGates + st * L::kGateBytes);
        const int valid = reinterpret_cast<const int32_t*>(gate)[257];
        // the exponents' high and low parts
        const float eh = gate[128 + t], el = gate[192 + t];
        const float2 eh2 = make_float2(eh, eh), el2 = make_float2(el, el);
        // the scores of the chunk before have been used
        if (it > 0 && !c.wait(L::kBars, L::bOFull, it - 1)) return;
        if (!c.wait(L::kBars, L::bPFull, it)) return;
        tc_fence_after();
        uint8_t* row = c.sm + L::kScores;
        if (!two) {
#pragma unroll
            for (int k = 0; k < L::kScoreParts; ++k)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    *reinterpret_cast<uint4*>(row + k * kPanel + sw128_off(t, empty / 8 + j)) = make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll 1
        for (int s = first; s < first + (two ? 32 : 16); s += 16) {
            float p[16];
            tmem_ld16w(c.tmem + lanes + L::tP + (L::kPSets == 2 ? (it & 1) * 64 : 0) + s, p);
#pragma unroll
            for (int j = 0; j < 16; j += 4) {
                const float4 sh = *reinterpret_cast<const float4*>(gate + 128 + s + j);
                const float4 sl = *reinterpret_cast<const float4*>(gate + 192 + s + j);
                const float2 d0 = add2(add2(eh2, make_float2(-sh.x, -sh.y)), add2(el2, make_float2(-sl.x, -sl.y)));
                const float2 d1 = add2(add2(eh2, make_float2(-sh.z, -sh.w)), add2(el2, make_float2(-sl.z, -sl.w)));
                const float d[4] = {d0.x, d0.y, d1.x, d1.y};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int at = s + j + e;
                    const bool keep = bw ? (at >= t && at < valid) : (at <= t);
                    p[j + e] = keep ? p[j + e] * exp2_fast(d[e]) : 0.f;
                }
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                uint32_t v[3][4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 x = make_float2(p[8 * j + 2 * e], p[8 * j + 2 * e + 1]);
                    if (kMode == kExact) split3(x, v[0][e], v[1][e], v[2][e]);
                    else split2(x, v[0][e], v[1][e]);
                }
#pragma unroll
                for (int k = 0; k < L::kScoreParts; ++k)
                    *reinterpret_cast<uint4*>(row + k * kPanel + sw128_off(t, s / 8 + j)) =
                        make_uint4(v[k][0], v[k][1], v[k][2], v[k][3]);
            }
        }
        // the product with z needs its rows behind the part's last token cleared too (the weights' warps clear them
        // for themselves; the same zeros)
        if (valid < kC) clear_rows(c.sm + st * L::kStage + L::kZ, valid);
        fence_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(c.bar(L::kBars, L::bPReady));
    }
}

// ---- warps 0-7: state -----------------------------------------------------------------------------------------
// Thread (quad, half, lane): row z = 32 quad + lane of the state, columns 64 half .. + 64.
template <int kMode>
GDN_DEVICE void put_state(const Ctx& c, uint32_t lanes, int half, const float* S) {
    using L = Layout<kMode>;
    const uint32_t dst = c.tmem + lanes + L::tA + half * 32;
#pragma unroll
    for (int j = 0; j < 64; j += 16) {
        uint32_t v[3][8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if (kMode == kExact) split3(make_float2(S[j + 2 * e], S[j + 2 * e + 1]), v[0][e], v[1][e], v[2][e]);
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

// A thread's 64 columns of a row, to and from a state in memory.  Transposed, lanes are neighbours there.  As it is,
// they are a row apart, and a warp's block of 32 rows x 64 columns goes through 8 KB of shared memory (16-byte pieces
// swizzled by the row) so that memory sees 256 bytes at a time; without room for that, row by row (6,000 cycles
// more for a state).
GDN_DEVICE float4* state_piece(uint8_t* buf, int row, int piece) {
    return reinterpret_cast<float4*>(buf + row * 256 + ((piece ^ (row & 15)) << 4));
}

GDN_DEVICE void load_state(float* S, const float* src, bool transposed, int z, int half, uint8_t* buf) {
    const int lane = threadIdx.x & 31;
    if (!src) {
#pragma unroll
        for (int j = 0; j < 64; ++j) S[j] = 0.f;
        return;
    }
    if (transposed) {
#pragma unroll
        for (int j = 0; j < 64; ++j) S[j] = src[(half * 64 + j) * kD + z];
        return;
    }
    if (buf) {
        const float* block = src + (z - lane) * kD + half * 64;
#pragma unroll 4
        for (int i = 0; i < 16; ++i) {
            const int row = 2 * i + (lane >> 4);
            *state_piece(buf, row, lane & 15) = *reinterpret_cast<const float4*>(block + row * kD + (lane & 15) * 4);
        }
        __syncwarp();
    }
#pragma unroll
    for (int j = 0; j < 64; j += 4) {
        const float4 v = buf ? *state_piece(buf, lane, j / 4) : *reinterpret_cast<const float4*>(src + z * kD + half * 64 + j);
        S[j] = v.x; S[j + 1] = v.y; S[j + 2] = v.z; S[j + 3] = v.w;
    }
}

GDN_DEVICE void store_state(const float* S, float* dst, bool transposed, int z, int half, uint8_t* buf) {
    const int lane = threadIdx.x & 31;
    if (transposed) {
#pragma unroll
        for (int j = 0; j < 64; ++j) dst[(half * 64 + j) * kD + z] = S[j];
        return;
    }
#pragma unroll
    for (int j = 0; j < 64; j += 4) {
        const float4 v = make_float4(S[j], S[j + 1], S[j + 2], S[j + 3]);
        if (buf) *state_piece(buf, lane, j / 4) = v;
        else *reinterpret_cast<float4*>(dst + z * kD + half * 64 + j) = v;
    }
    if (buf) {
        __syncwarp();
        float* block = dst + (z - lane) * kD + half * 64;
#pragma unroll 4
        for (int i = 0; i < 16; ++i) {
            const int row = 2 * i + (lane >> 4);
            *reinterpret_cast<float4*>(block + row * kD + (lane & 15) * 4) = *state_piece(buf, row, lane & 15);
        }
        __syncwarp();
    }
}

template <int kMode>
GDN_DEVICE void state_role(const Ctx& c) {
    using L = Layout<kMode>;
    const LinPass& p = c.w.p;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, quad = warp & 3, half = warp >> 2;
    const int z = quad * 32 + lane;
    const uint32_t lanes = (uint32_t)(quad * 32) << 16;
    float S[64];
    Ring<L::kStages> ring;
    constexpr int kKvSets = L::kKvSets;
    uint32_t it = 0;
    for (int r = 0; r < c.reps; ++r) {
        const int h = c.head0 + r;
        const int64_t own = ((int64_t)c.part.seq * p.Hv + h) * (kD * kD);
        const int64_t joint = ((int64_t)c.part.slot * p.Hv + h) * (kD * kD);
        // kOut: the last stage, which the loads leave alone until then
        uint8_t* room = kMode == kOut && r == 0 ? c.sm + (L::kStages - 1) * L::kStage + warp * 8192 : nullptr;
        if (kMode == kState) load_state(S, nullptr, false, z, half, nullptr);
        else if (c.w.split && !c.part.alone) load_state(S, c.w.joint + joint, c.w.joint_t != 0, z, half, room);
        else load_state(S, p.init ? p.init + own : nullptr, p.state_t != 0, z, half, room);
        if (kMode == kOut && r == 0) {
            fence_async_smem();                 // every lane's last access to the room comes before TMA's writes there
            __syncwarp();
            if (lane == 0) mbar_arrive(c.bar(L::kBars, L::bStateIn));
        }
        // turn n: the state behind chunk n - 1, and its copy for chunk n
#pragma unroll 1
        for (int32_t n = 0; n <= c.chunks; ++n) {
            if (n > 0) {
                const float* gate = reinterpret_cast<const float*>(c.sm + L::kGates + ring.st * L::kGateBytes);
                if (!c.wait(L::kBars, L::bFull + ring.st, ring.phase)) return;
                const float2 gamma2 = make_float2(gate[256], gate[256]);
                if (!c.template wait_set<kKvSets>(L::kBars, L::bKvFull, it)) return;
                tc_fence_after();
                const uint32_t set = kKvSets == 2 ? it & 1u : 0u;
#pragma unroll
                for (int j = 0; j < 64; j += 32) {
                    float kv[32];
                    tmem_ld32w(c.tmem + lanes + L::tKv + set * 128 + half * 64 + j, kv);
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        const float2 x = fma2(gamma2, make_float2(S[j + e], S[j + e + 1]), make_float2(kv[e], kv[e + 1]));
                        S[j + e] = x.x;
                        S[j + e + 1] = x.y;
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(c.bar(L::kBars, L::bKvFree + set));
                    mbar_arrive(c.bar(L::kBars, L::bEmpty + ring.st));
                }
                ring.next();
                // inter has read the copy for the chunk before
                if (L::kOuts) {
                    if (!c.wait(L::kBars, L::bOFull, it)) return;
                    tc_fence_after();
                }
                ++it;
            }
            if (L::kOuts && n < c.chunks) put_state<kMode>(c, lanes, half, S);
        }
        // After the last head's last chunk nothing is loaded any more.  kState: the products are done with every stage.
        // kOut: and so is the output with the stage after the last chunk's, that of the third last chunk (its rows had
        // left before the second last chunk's inter and intra were released, which the last chunk's products needed).
        room = r + 1 == c.reps && kMode != kExact ? c.sm + (kMode == kOut ? ring.st * L::kStage : 0) + warp * 8192 : nullptr;
        if (kMode == kState) store_state(S, c.w.joint + joint, false, z, half, room);
        else if (p.fin && c.part.last) store_state(S, p.fin + own, p.state_t != 0, z, half, room);
    }
}

// NaN in this warp's staged output, from the first token on whose z is not finite, and in its part of the dot products
template <int kMode>
GDN_DEVICE void put_nan(const Ctx& c, int st, int buf, uint32_t rows, int quad, int half, int lane, bool f32) {
    using L = Layout<kMode>;
    const bool bw = c.w.p.backward != 0;
    const int z = quad * 32 + lane, at = reinterpret_cast<const int32_t*>(c.sm + L::kBad + st * 512)[z] - half * 32;
    uint8_t* to = c.sm + st * L::kStage + rows;
    __syncwarp();                               // the warp's output is in place
#pragma unroll 1
    for (int t = 0; t < 32; ++t) {
        const bool here = bw ? t <= at : t >= at;
        if (here && f32) *reinterpret_cast<uint32_t*>(to + quad * L::kRows + sw128_off(t, lane >> 2) + (lane & 3) * 4) = 0x7fc00000u;
        if (here && !f32) *reinterpret_cast<uint16_t*>(to + (z >> 6) * L::kRows + sw128_off(t, (z & 63) >> 3) + (z & 7) * 2) = 0x7fc0u;
        if (kMode == kExact && __any_sync(0xffffffffu, here) && lane == 0)
            reinterpret_cast<uint32_t*>(c.sm + L::kDots)[buf * 256 + (half * 4 + quad) * 32 + t] = 0x7fc00000u;
    }
}

// ---- warps 8-15: output -----------------------------------------------------------------------------------------
// Warp (quad, half): z indices 32 quad .. + 32, tokens 32 half .. + 32.
template <int kMode>
GDN_DEVICE void out_role(const Ctx& c, const CUtensorMap* mo) {
    using L = Layout<kMode>;
    const LinPass& p = c.w.p;
    const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) - 8, quad = warp & 3, half = warp >> 2;
    const uint32_t lanes = (uint32_t)(quad * 32) << 16;
    const int heads = p.Hv / p.out_rep;
    const float2 fa2 = p.backward ? make_float2(1.f, 1.f) : make_float2(p.scale, p.scale);
    const float2 fp2 = make_float2(p.scale, p.scale);
    const bool f32 = p.out_rep > 1 || !p.out_bf16;
    const uint32_t rows = L::kHalf * half;      // of a stage: where the output is staged, over x, whose products are done
    Ring<L::kStages> ring;
    uint32_t it = 0;
    int held = -1;                              // the stage whose rows are leaving
    for (int r = 0; r < c.reps; ++r) {
#pragma unroll 1
        for (int32_t n = 0; n < c.chunks; ++n) {
            const int st = ring.st;
            const float* gate = reinterpret_cast<const float*>(c.sm + L::kGates + st * L::kGateBytes);
            if (!c.wait(L::kBars, L::bFull + st, ring.phase)) return;
            const int64_t t0 = c.chunk_start(n);
            const int valid = reinterpret_cast<const int32_t*>(gate)[257];
            if (!c.wait(L::kBars, L::bOFull, it)) return;
            const uint32_t set = L::kPSets == 2 ? it & 1u : 0u;
            const bool bad = reinterpret_cast<const uint32_t*>(gate)[L::kFlags / 4 + quad] != 0u;
            tc_fence_after();
            if (held >= 0 && lane == 0) {       // the chunk before's rows have left its stage
                bulk_wait_read();
                mbar_arrive(c.bar(L::kBars, L::bEmpty + held));
            }
            held = -1;
            // The fragment layout of transposed 8 x 8 matrices: tokens tq + 8 j (+ 1), z indices 32 quad + 16 hz +
            // lane / 4 (+ 8)
            const int tq = 2 * (lane & 3);
            const uint32_t stage = c.base + st * L::kStage;
            uint32_t at32[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) at32[e] = sw128_off(tq + e, lane >> 4) + ((lane >> 2) & 3) * 4;
            // matrix m of 16 tokens and 16 z indices: tokens 8 (m >> 1), z indices 8 (m & 1)
            const int mt = ((lane >> 4) << 3) + (lane & 7), mz = quad * 32 + ((lane >> 3) & 1) * 8;
#pragma unroll 1
            for (int tb = 0; tb < 32; tb += 16) {
                const float2 a0 = mul2(fa2, *reinterpret_cast<const float2*>(gate + half * 32 + tb + tq));
                const float2 a1 = mul2(fa2, *reinterpret_cast<const float2*>(gate + half * 32 + tb + tq + 8));
                float dot[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
                for (int hz = 0; hz < 32; hz += 16) {
                    float inter[8], out[8];
                    const uint32_t src = c.tmem + lanes + ((uint32_t)hz << 16) + half * 32 + tb;
                    tmem_ld_frag16x2w(src + L::tInter, src + L::tP + set * 64, inter, out);
                    if (tb + hz == 32) {        // the last of this warp's: the products may go on
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(c.bar(L::kBars, L::bOFree));
                    }
#pragma unroll
                    for (int e = 0; e < 8; e += 2) {
                        const float2 x = fma2(e < 4 ? a0 : a1, make_float2(inter[e], inter[e + 1]),
                                              mul2(fp2, make_float2(out[e], out[e + 1])));
                        out[e] = x.x;
                        out[e + 1] = x.y;
                    }
                    const int zm = mz + hz, tm = tb + mt;               // this lane's row of a matrix, of the half
                    if (kMode == kExact) {
                        uint32_t u[4];
                        ldmatrix_x4_trans(stage + L::kU + (zm >> 6) * kPanel + sw128_off(half * 32 + tm, (zm & 63) >> 3), u);
#pragma unroll
                        for (int m = 0; m < 4; ++m) {
                            const float2 f = bf16x2_to_f32x2(u[m]);
                            const int g = m >> 1;                       // the 8-token group
                            dot[2 * g] = fmaf(f.x, out[2 * m], dot[2 * g]);
                            dot[2 * g + 1] = fmaf(f.y, out[2 * m + 1], dot[2 * g + 1]);
                        }
                    }
                    if (f32) {
                        // row tb + tq + 8 (e / 4) + e % 2, element hz + 8 (e / 2 % 2) + lane / 4 of the quadrant's 32: its
                        // 16-byte piece is swizzled by the row, so a warp's rows put theirs in different places
                        uint8_t* to = c.sm + st * L::kStage + rows + quad * L::kRows + tb * 128;
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            *reinterpret_cast<float*>(to + (e >> 2) * 1024 + (at32[e & 1] ^ (((e >> 1) & 1) << 5) ^ (hz << 2))) = out[e];
                    } else {
                        uint32_t v[4];
#pragma unroll
                        for (int m = 0; m < 4; ++m) v[m] = pack_bf16x2(out[2 * m], out[2 * m + 1]);
                        stmatrix_x4_trans(stage + rows + (zm >> 6) * L::kRows + sw128_off(tm, (zm & 63) >> 3), v);
                    }
                }
                if (kMode == kExact) {
                    // u_t . out_t over this warp's 32 z indices: lanes of one lane % 4 hold the same tokens; lanes
                    // m apart exchange the half of their sums that the other one keeps
                    const float g0 = lane & 4 ? dot[0] : dot[2], g1 = lane & 4 ? dot[1] : dot[3];
                    float k0 = lane & 4 ? dot[2] : dot[0], k1 = lane & 4 ? dot[3] : dot[1];
                    k0 += __shfl_xor_sync(0xffffffffu, g0, 4);
                    k1 += __shfl_xor_sync(0xffffffffu, g1, 4);
                    const float g2 = lane & 8 ? k0 : k1;
                    float k2 = lane & 8 ? k1 : k0;
                    k2 += __shfl_xor_sync(0xffffffffu, g2, 8);
                    k2 += __shfl_xor_sync(0xffffffffu, k2, 16);
                    if (lane < 16)
                        reinterpret_cast<float*>(c.sm + L::kDots)[(it & 1u) * 256 + warp * 32 + tb + (lane & 4) * 2 +
                                                                  2 * (lane & 3) + (lane >> 3)] = k2;
                }
            }
            if (bad) put_nan<kMode>(c, st, (int)(it & 1u), rows, quad, half, lane, f32);
            fence_async_smem();
            const bool whole = half * 32 + 32 <= valid;         // every row of this half is this part's
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(c.bar(L::kBars, L::bRows + half + 2 * (int)(it & 1u)));
                if (whole && quad != 0) mbar_arrive(c.bar(L::kBars, L::bEmpty + st));
            }
            const uint32_t now = it++;
            ring.next();
            if (whole && quad != 0) continue;
            // The four warps of this half have their z indices in place.  Two barriers in turn: a warp that has not yet
            // arrived for this chunk has released its products all the same, so the others may arrive for the next one
            // before it (not for the one after, whose products wait for all of them).
            if (!c.wait(L::kBars, L::bRows + half + 2 * (int)(now & 1u), now >> 1)) return;
            if (kMode == kExact && quad == 0 && half * 32 + lane < valid) {
                // (two buffers: the chunk after the next needs this stage, which this warp has not yet released)
                static_assert(kMode != kExact || L::kStages == 2, "the buffers of the dot products");
                const float* d = reinterpret_cast<const float*>(c.sm + L::kDots) + (now & 1u) * 256 + half * 128 + lane;
                p.dots[(int64_t)(c.head0 + r) * p.T + t0 + half * 32 + lane] = (d[0] + d[32]) + (d[64] + d[96]);
            }
            __syncwarp();
            if (whole) {
                if (lane == 0) {
                    const int32_t x = c.head * kD, y = (int32_t)t0 + half * 32;
                    const uint32_t from = stage + rows;
                    if (!f32) {
                        tma_store_2d(mo, x, y, from);
                        tma_store_2d(mo, x + 64, y, from + L::kRows);
                    } else {
#pragma unroll 1
                        for (int k = 0; k < 4; ++k) {
                            if (r == 0) tma_store_2d(mo, x + 32 * k, y, from + k * L::kRows);
                            else tma_add_2d(mo, x + 32 * k, y, from + k * L::kRows);
                        }
                    }
                    bulk_commit();
                    if (kMode == kExact) {
                        // With two stages the next but one chunk's loads wait for these rows to leave: at once, not
                        // at the next turn (7,100 cycles a chunk).
                        bulk_wait_read();
                        mbar_arrive(c.bar(L::kBars, L::bEmpty + st));
                    }
                }
                if (kMode != kExact) held = st;
            } else {
                // the part's last rows: those behind them are not this part's, so plain stores, 8 rows a warp
                const int pieces = f32 ? 32 : 16;
                float* o32 = p.out_bf16 ? p.acc : static_cast<float*>(p.out);
#pragma unroll 1
                for (int i = lane; i < 8 * pieces; i += 32) {
                    const int row = quad * 8 + i / pieces, piece = i % pieces;
                    if (half * 32 + row >= valid) break;
                    const int64_t at = ((t0 + half * 32 + row) * heads + c.head) * kD;
                    uint4 v = *reinterpret_cast<const uint4*>(c.sm + st * L::kStage + rows + (piece >> 3) * L::kRows +
                                                              sw128_off(row, piece & 7));
                    if (!f32) {
                        reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + at)[piece] = v;
                    } else {
                        float4* to = reinterpret_cast<float4*>(o32 + at) + piece;
                        float4 x = make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z), __uint_as_float(v.w));
                        if (r > 0) {
                            const float4 y = *to;
                            x = make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
                        }
                        *to = x;
                    }
                }
            }
            __syncwarp();
            if (!whole && lane == 0) mbar_arrive(c.bar(L::kBars, L::bEmpty + st));
        }
        // this head's rows are in place before the next head adds to them
        bulk_wait();
    }
}

template <int kMode, int kPasses>
__global__ void __launch_bounds__(kThreads, 1)
lin_walk_kernel(const __grid_constant__ Passes<kPasses> passes) {
    using L = Layout<kMode>;
    const int which = kPasses == 2 && (int32_t)blockIdx.x >= passes.blocks ? 1 : 0;
    const unsigned block = blockIdx.x - (unsigned)which * passes.blocks;       // of its pass
    const Walk& w = passes.w[which];
    extern __shared__ uint8_t raw[];
    uint8_t* sm = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
    const uint32_t base = smem_u32(sm);
    const int warp = threadIdx.x >> 5;
    const int heads = kMode == kState ? w.p.Hv : w.p.Hv / w.p.out_rep;
    const int32_t index = (int32_t)(block / heads);
    // (well before any CTA can have waited long enough to raise it)
    if (w.opens && blockIdx.x == 0 && threadIdx.x == 0) *w.err = 0u;
    if (w.part_seq) grid_wait();                // the lists come from a kernel before
    const Part part = find_part(w, index, kMode == kState);       // (the last part's own sum is not needed)
    if (part.seq < 0) {
        grid_wait();
        return;
    }
    volatile int* abort = reinterpret_cast<volatile int*>(sm + L::kMisc + 8);
    if (threadIdx.x == 0) {
        auto init = [&](int i, uint32_t n) { mbar_init(base + L::kBars + i * 8, n); };
        for (int s = 0; s < L::kStages; ++s) {
            init(L::bFull + s, 2);                  // the loads' bytes; the decays
            init(L::bEmpty + s, kMode == kState ? 1 + 8 : 2 + 8 + 8);       // the products; warps 0-7; warps 8-15
        }
        init(L::bPFull, 1);
        init(L::bPReady, 4);
        init(L::bAReady, 8);
        for (int k = 0; k < 2; ++k) {
            init(L::bKvFull + k, 1);
            init(L::bKvFree + k, 8);
        }
        init(L::bOFull, 1);
        init(L::bOFree, 8);
        for (int k = 0; k < L::kSlotBufs; ++k) {
            init(L::bWFull + k, 4);
            init(L::bWFree + k, 1);
        }
        init(L::bZeroed, kMode == kState ? 8 : 4);
        for (int k = 0; k < 4; ++k) init(L::bRows + k, 4);
        init(L::bDrain, 1);
        init(L::bDrain + 1, 1);
        init(L::bDone, 27);
        init(L::bStateIn, 8);
        for (int k = 0; k < 4; ++k) init(L::bZDone + k, 4);
        *abort = 0;
        fence_mbar_init();
    }
    if (warp == 25) tmem_alloc(base + L::kMisc, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    grid_wait();
    grid_next();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(sm + L::kMisc);
    const int head = (int)(block - (unsigned)index * heads);
    const int reps = kMode == kState ? 1 : w.p.out_rep;
    const Ctx c{w, sm, base, tmem, abort, base + L::kMisc + 8, part, (int32_t)((part.t1 - part.t0 + kC - 1) / kC), head, reps, head * reps};
    if (warp < 8) {
        regs_inc<kRegsState>();
        state_role<kMode>(c);
    } else if (warp < 16) {
        regs_dec<kRegsOut>();
        if (L::kOuts) out_role<kMode>(c, &passes.out[which]);
        else if (warp == 8) decay_role<kMode>(c, 1, 2);
        bulk_wait();                            // rows still leaving (a role that gave up)
    } else if (warp < 20) {
        weight_role<kMode>(c, 0, kMode == kState ? 2 : 1);
    } else if (warp < 24) {
        regs_dec<kRegsScores>();
        if (kMode == kState) weight_role<kMode>(c, 1, 2);
        else score_role<kMode>(c);
    } else {
        regs_dec<kRegsRest>();
        if (warp == 24) load_role<kMode>(c, &passes.x[which], &passes.y[which], &passes.z[which], &passes.u[which]);
        if (warp == 25) kv_role<kMode>(c, 0);
        if (warp == 26 && L::kOuts) out_products_role<kMode>(c);
        if (warp == 26 && kMode == kState) kv_role<kMode>(c, 1);
        if (warp == 27) {
            decay_role<kMode>(c, 0, kMode == kState ? 2 : 1);
            mbar_wait(c.bar(L::kBars, L::bDone), 0, c.abort, kWaitLimitNs);
        }
    }
    if (warp != 27) {
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive(base + L::kBars + L::bDone * 8);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (*abort && threadIdx.x == 0) *w.err = 1u;
    if (kMode == kState && threadIdx.x == 0) {
        // the part's whole decay
        const long long* sum = reinterpret_cast<const long long*>(sm + L::kMisc + 16);
        const float* bad = reinterpret_cast<const float*>(sm + L::kMisc + 32);
        w.joint_decay[(int64_t)part.slot * w.p.Hv + head] =
            exp2f((float)((double)(sum[0] + sum[1]) * (1.0 / 4294967296.0))) + bad[0] + bad[1];
    }
    tc_fence_after();
    if (warp == 25) tmem_dealloc(tmem, 512);
}

}  // namespace lin
}  // namespace gdn
