// linear_decode.cu -- one token of linear attention with a decay per head for
// many (sequence, layer) units, the state updated in place:
//     S <- e^g S + v k^T,   o = scale S q.
// Row i of S changes as S_i <- e^g S_i + v_i k and gives o_i = scale S_i . q,
// so every row is read once and written once and the step is bound by HBM
// bandwidth (2 x 64 KiB per value head in float32, half of it in bf16).  The
// decayed element is rounded to float32 before the product v_i k_j, which
// float32 holds exactly, is added: the two operations of the definition, so that
// a bf16 state rounds as theirs does, step after step.
//
// Mapping: 128 threads per (unit, value head), or per part of its rows (below).
// A lane holds 16 bytes of a row, so a float32 row is one warp's access and two
// bf16 rows are; eight accesses per lane are in flight.  The dot products of
// those rows are reduced together: at each step lanes m apart exchange the
// half of their sums that the other one keeps, 8 + 2 shuffles where one row at
// a time takes 40.
//
// Measured: 64 sequences x 48 layers x 48 heads, bf16 state, 9.2 GB in 1.43 ms, 97%
// of the measured copy rate; one sequence of 4 layers x 12 heads 4.3 us.
//
// With few (unit, head) pairs a CTA per pair leaves SMs idle and walks its rows
// in four rounds; each pair is then split over up to 4 CTAs by rows, which
// share nothing but q and k.
#include "common.cuh"
#include "kernels.h"

namespace gdn {

namespace {

constexpr int kD = 128;
constexpr int kThreads = 128;
constexpr int kLoads = 8;                       // 16-byte accesses in flight per lane

// 16 bytes of a state row <-> float32
template <typename StateT>
struct Row;
template <>
struct Row<float> {
    static constexpr int kCols = 4;             // of a lane
    static GDN_DEVICE void unpack(const uint4& r, float* x) {
        x[0] = __uint_as_float(r.x); x[1] = __uint_as_float(r.y);
        x[2] = __uint_as_float(r.z); x[3] = __uint_as_float(r.w);
    }
    static GDN_DEVICE uint4 pack(const float* x) {
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
    }
};
template <>
struct Row<uint16_t> {
    static constexpr int kCols = 8;
    static GDN_DEVICE void unpack(const uint4& r, float* x) {
        float2 f;
        f = bf16x2_to_f32x2(r.x); x[0] = f.x; x[1] = f.y;
        f = bf16x2_to_f32x2(r.y); x[2] = f.x; x[3] = f.y;
        f = bf16x2_to_f32x2(r.z); x[4] = f.x; x[5] = f.y;
        f = bf16x2_to_f32x2(r.w); x[6] = f.x; x[7] = f.y;
    }
    // the state is rounded to bf16 (nearest even) only when it is stored
    static GDN_DEVICE uint4 pack(const float* x) {
        return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                          pack_bf16x2(x[6], x[7]));
    }
};

template <int kCols>
GDN_DEVICE void load_cols(const uint16_t* p, float* x) {
#pragma unroll
    for (int c = 0; c < kCols; c += 4) {
        const uint2 b = *reinterpret_cast<const uint2*>(p + c);
        float2 f;
        f = bf16x2_to_f32x2(b.x); x[c] = f.x; x[c + 1] = f.y;
        f = bf16x2_to_f32x2(b.y); x[c + 2] = f.x; x[c + 3] = f.y;
    }
}

template <typename StateT>
__global__ void __launch_bounds__(kThreads, 5) linear_decode_kernel(LinearDecodeArgs a, int splits) {
    using R = Row<StateT>;
    constexpr int kCols = R::kCols;
    constexpr int kLanes = kD / kCols;          // lanes of a row
    constexpr int kRows = 32 / kLanes;          // rows of a warp's access
    constexpr int kBatch = kLoads * kRows;      // rows of a warp's round
    const int64_t uh = (int64_t)blockIdx.x / splits;
    const int part = (int)(blockIdx.x - uh * splits);
    const int64_t unit = uh / a.Hv;             // sequence * layers + layer
    const int h = (int)(uh - unit * a.Hv);
    const int64_t n = unit / a.layers;
    const int l = (int)(unit - n * a.layers);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t slot = a.slot ? a.slot[n] : n;
    const int rows = kD / splits;               // of this CTA
    if (slot < 0 || slot >= a.n_slots) {        // a row without a sequence: no state, a zero output
        const int i = part * rows + threadIdx.x;
        if (threadIdx.x < rows) {
            if (a.o_bf16) static_cast<uint16_t*>(a.o)[uh * kD + i] = 0;
            else static_cast<float*>(a.o)[uh * kD + i] = 0.f;
        }
        return;
    }
    StateT* S = static_cast<StateT*>(a.state) + ((slot * a.layers + l) * a.Hv + h) * (int64_t)(kD * kD);
    const int64_t qk = (unit * a.Hqk + h / (a.Hv / a.Hqk)) * kD;
    const int col = (lane % kLanes) * kCols, sub = lane / kLanes;
    float q[kCols], k[kCols];
    load_cols<kCols>(a.q + qk + col, q);
    load_cols<kCols>(a.k + qk + col, k);
    const float decay = expf(a.g[(a.g_per_unit ? unit : (int64_t)l) * a.Hv + h]);
    const uint16_t* v = a.v + uh * kD;
    const int per_warp = rows / 4;              // 32, 16 or 8
    const int first = part * rows + warp * per_warp;

    for (int r0 = first; r0 < first + per_warp; r0 += kBatch) {
        uint4 raw[kLoads];
        float vr[kLoads], dot[kLoads];
        const int here = min(kBatch, first + per_warp - r0) / kRows;       // accesses of this round
#pragma unroll
        for (int j = 0; j < kLoads; ++j)
            if (j < here) raw[j] = __ldcs(reinterpret_cast<const uint4*>(S + (int64_t)(r0 + j * kRows + sub) * kD + col));
#pragma unroll
        for (int j = 0; j < kLoads; ++j) vr[j] = j < here ? bf16_to_f32(v[r0 + j * kRows + sub]) : 0.f;
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            dot[j] = 0.f;
            if (j < here) {
                float s[kCols];
                R::unpack(raw[j], s);
#pragma unroll
                for (int c = 0; c < kCols; ++c) {
                    s[c] = fmaf(vr[j], k[c], __fmul_rn(decay, s[c]));
                    dot[j] = fmaf(s[c], q[c], dot[j]);
                }
                __stcs(reinterpret_cast<uint4*>(S + (int64_t)(r0 + j * kRows + sub) * kD + col), R::pack(s));
            }
        }
        // after the three exchanges a lane holds the sum of one access (index lane & 7 in bit-reversed order)
#pragma unroll
        for (int m = 1, half = kLoads / 2; half >= 1; m <<= 1, half >>= 1)
#pragma unroll
            for (int j = 0; j < half; ++j) {
                const float give = (lane & m) ? dot[j] : dot[j + half];
                const float keep = (lane & m) ? dot[j + half] : dot[j];
                dot[j] = keep + __shfl_xor_sync(0xffffffffu, give, m);
            }
#pragma unroll
        for (int m = kLoads; m < kLanes; m <<= 1) dot[0] += __shfl_xor_sync(0xffffffffu, dot[0], m);
        const int j = ((lane & 1) << 2) | (lane & 2) | ((lane & 4) >> 2);
        if (lane % kLanes < kLoads && j < here) {
            const int64_t at = uh * kD + r0 + j * kRows + sub;
            const float o = a.scale * dot[0];
            if (a.o_bf16) static_cast<uint16_t*>(a.o)[at] = (uint16_t)f32_to_bf16_bits(o);
            else static_cast<float*>(a.o)[at] = o;
        }
    }
}

}  // namespace

cudaError_t launch_linear_decode(const LinearDecodeArgs& a, cudaStream_t stream) {
    const int64_t pairs = (int64_t)a.n_seq * a.layers * a.Hv;
    if (pairs == 0) return cudaSuccess;
    // rows split over CTAs while that still fills no more than one round of 5 CTAs on 148 SMs
    const int splits = pairs * 4 <= 740 ? 4 : pairs * 2 <= 740 ? 2 : 1;
    if (pairs * splits > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    const unsigned blocks = (unsigned)(pairs * splits);
    if (a.state_bf16) linear_decode_kernel<uint16_t><<<blocks, kThreads, 0, stream>>>(a, splits);
    else linear_decode_kernel<float><<<blocks, kThreads, 0, stream>>>(a, splits);
    return cudaGetLastError();
}

}  // namespace gdn
