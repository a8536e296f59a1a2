// linear_walk.cu -- launches of the linear attention passes (linear_walk.cuh):
// the prefill is one pass, its gradients are three (linear_attn.h).
#include <cuda.h>

#include <atomic>

#include "launch_chain.h"
#include "linear_walk.cuh"

namespace gdn {

namespace {

using namespace lin;

constexpr int kSms = 148;

size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

// ---- parts --------------------------------------------------------------------------------------------
// The length of a part, from what the host knows: T tokens in n_seq sequences, of which it assumes equal lengths
// where it cuts them, and one of eight times the mean where it leaves them whole.  The least of
//     walk:    rounds of `heads` CTAs per part over the SMs, each reps * chunks * kWalk + kStart long
//     states:  where a sequence has several parts, the same over all parts but the last, chunks * kStateStep long,
//              and the scan
// in microseconds, measured on B200.  Sequences that turn out longer than a part are cut.  Only lengths for which the
// workspace suffices (`fits`) count; the longest there is needs the least.
template <typename Fits>
int32_t choose_part_len(int32_t n_seq, int64_t T, int32_t heads, int32_t reps, int64_t most, const Fits& fits) {
    constexpr double kWalk = 2.1, kStateStep = 0.85, kStart = 5.0, kScan = 8.0;
    const int64_t all = (T + kC - 1) / kC, chunks = (T + n_seq - 1) / n_seq / kC + 1;
    auto rounds = [](int64_t ctas) { return (double)((ctas + kSms - 1) / kSms); };
    double best = -1.0;
    int64_t len = most / kC;
    if (T <= most) {
        best = rounds((int64_t)n_seq * heads) * kStart + (rounds((int64_t)n_seq * heads) - 1) * (double)(chunks * reps) * kWalk +
               (double)((all < 8 * chunks ? all : 8 * chunks) * reps) * kWalk;
        len = all > 0 ? all : 1;
    }
    for (int64_t parts = 1; parts <= chunks && parts <= kSms; ++parts) {
        const int64_t l = (chunks + parts - 1) / parts;
        if (l * kC > most || l >= all) continue;
        const int64_t n = (chunks + l - 1) / l;
        double cost = rounds((int64_t)n_seq * n * heads) * ((double)(l * reps) * kWalk + kStart);
        // (uneven sequences are cut even where their mean is not)
        cost += rounds((int64_t)n_seq * (n > 1 ? n - 1 : 1) * heads * reps) * ((double)l * kStateStep + kStart) + kScan;
        const int64_t whole = n == 1 && 2 * l * kC <= most ? 2 * l : l;            // up to twice the mean stays whole
        if ((best < 0.0 || cost < best) && fits((int32_t)(whole * kC))) {
            best = cost;
            len = whole;
        }
    }
    return (int32_t)(len * kC);
}

int32_t part_count(int32_t n_seq, int64_t T, int32_t part_len) { return (int32_t)(T / part_len) + n_seq; }

// Turns each part's own sum into its starting state: start' = decay * start + own along the parts of a
// sequence, in the pass's direction, from init.  One CTA per (sequence, head, 1024 elements).  Bound by the latency
// of its loads, four parts' at a time (9 parts of 48 heads: 7.5 us, the sums still in L2).
constexpr int kScanThreads = 256;
constexpr int kScanSeqs = 32;                  // sequences at a time

GDN_DEVICE void scan_sequence(const Walk& w, int seq, int h, int e) {
    int32_t before = 0, n;
    if (w.part_seq) {
        before = w.seq_first[seq];
        n = w.seq_first[seq + 1] - before;
    } else {                                    // (at most 32 sequences)
        auto parts = [&](int i) {
            return parts_of(w, w.p.cu ? w.p.cu[i] : 0, w.p.cu ? w.p.cu[i + 1] : (int32_t)w.p.T);
        };
        n = parts(seq);
        for (int i = 0; i < seq; ++i) before += parts(i);
    }
    if (n == 1) return;
    auto slot = [&](int k) { return (int64_t)(before + (w.p.backward ? n - 1 - k : k)) * w.p.Hv + h; };
    float4 run = make_float4(0.f, 0.f, 0.f, 0.f);
    if (w.p.init) run = *reinterpret_cast<const float4*>(w.p.init + ((int64_t)seq * w.p.Hv + h) * (kD * kD) + e);
    constexpr int kBatch = 4;                   // parts whose sums are in flight at once
    for (int k0 = 0; k0 < n; k0 += kBatch) {
        float4 own[kBatch];
        float decay[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
            if (k0 + k < n - 1) {
                own[k] = *reinterpret_cast<const float4*>(w.joint + slot(k0 + k) * (kD * kD) + e);
                decay[k] = w.joint_decay[slot(k0 + k)];
            }
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
            if (k0 + k < n) {
                *reinterpret_cast<float4*>(w.joint + slot(k0 + k) * (kD * kD) + e) = run;
                if (k0 + k < n - 1) {
                    run.x = fmaf(decay[k], run.x, own[k].x);
                    run.y = fmaf(decay[k], run.y, own[k].y);
                    run.z = fmaf(decay[k], run.z, own[k].z);
                    run.w = fmaf(decay[k], run.w, own[k].w);
                }
            }
    }
}

__global__ void __launch_bounds__(kScanThreads) lin_scan_kernel(const __grid_constant__ WalkPair pair) {
    const Walk& w = pair.w[blockIdx.z];
    grid_wait();
    grid_next();
    const int h = blockIdx.x % w.p.Hv;
    for (int seq = blockIdx.x / w.p.Hv; seq < w.p.n_seq; seq += kScanSeqs)
        scan_sequence(w, seq, h, (blockIdx.y * kScanThreads + threadIdx.x) * 4);
}

// The parts of many sequences, written out (Walk's lists).  One CTA.
constexpr int kListThreads = 1024;

__global__ void __launch_bounds__(kListThreads)
lin_parts_kernel(const __grid_constant__ Walk w, int32_t* part_seq, int32_t* inner, int32_t* seq_first) {
    __shared__ int32_t sums[kListThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    grid_wait();
    grid_next();
    if (tid == 0) *w.err = 0u;
    for (int32_t i = tid; i < w.n_parts; i += kListThreads) part_seq[i] = -1;
    for (int32_t i = tid; i < w.n_inner; i += kListThreads) inner[i] = -1;
    __syncthreads();
    int32_t before = 0;                         // parts of the sequences in front of this block's
    for (int32_t i0 = 0; i0 < w.p.n_seq; i0 += kListThreads) {
        const int32_t i = i0 + tid;
        const int32_t n = i < w.p.n_seq ? parts_of(w, w.p.cu[i], w.p.cu[i + 1]) : 0;
        int32_t upto = n;
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const int32_t x = __shfl_up_sync(0xffffffffu, upto, m);
            if (lane >= m) upto += x;
        }
        if (lane == 31) sums[warp] = upto;
        __syncthreads();
        int32_t all = 0;
        for (int k = 0; k < kListThreads / 32; ++k) {
            if (k < warp) upto += sums[k];
            all += sums[k];
        }
        __syncthreads();
        if (i < w.p.n_seq) {
            const int32_t first = before + upto - n;
            seq_first[i] = first;
            if (i + 1 == w.p.n_seq) seq_first[i + 1] = first + n;
            for (int32_t k = 0; k < n; ++k) part_seq[first + k] = i;
            for (int32_t k = 0; k + 1 < n; ++k) inner[first - i + k] = first + k;
        }
        before += all;
    }
}

// The decays' gradient (linear_attn.h's passes give r_t = q_t . dq_t and c_t = k_t . dk_t): with S and dS the
// state and its gradient behind token t,
//     dg_t = <S_end, dS_end> + sum_{t' >= t, same part} (r_t' - c_t'),
// the first term at the part's end from the joints (or the final state), the sums in 64 bits from the last
// token back.  The sum at the part's first token is known too, <S, dS> in front of it: what the float32 errors of
// r and c have added up to by then is taken back in proportion to the tokens summed, which leaves about 0.6 of the
// error (a random walk tied down at both ends).  One CTA per (part, head).  Bound by the chain of its blocks' sums (8,192
// tokens of 48 heads: 26 us).
constexpr int kDgThreads = 256;

GDN_DEVICE double block_sum(double x, double* sm) {
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
    if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = x;
    __syncthreads();
    double s = 0.0;
    for (int i = 0; i < kDgThreads / 32; ++i) s += sm[i];
    __syncthreads();
    return s;
}

// <a, b> of two states, 0 if one is NULL: 16 products to a float32 sum, whose rounding is that of the states'
// elements themselves, the sums' sum in 64 bits (all of it in 64 bits took the kernel 31 us at 8,192 tokens)
GDN_DEVICE double state_product(const float* a, const float* b, double* sm) {
    if (!a || !b) return 0.0;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int i = threadIdx.x * 4; i < kD * kD; i += kDgThreads * 4) {
        const float4 x = *reinterpret_cast<const float4*>(a + i), y = *reinterpret_cast<const float4*>(b + i);
        s = make_float4(fmaf(x.x, y.x, s.x), fmaf(x.y, y.y, s.y), fmaf(x.z, y.z, s.z), fmaf(x.w, y.w, s.w));
    }
    return block_sum(((double)s.x + s.y) + ((double)s.z + s.w), sm);
}

struct DgArgs {
    const float* r;
    const float* c;
    const float* joint_end;         // dS at the parts' ends
    const float* fin;               // the final states and their gradients, or NULL
    const float* d_fin;
    const float* d_init;            // the initial states' gradients, or NULL (the states: Walk's init)
    float* dg;
    double* part_sum;               // for shared decays: the parts' sums instead of dg
};

__global__ void __launch_bounds__(kDgThreads)
lin_dg_kernel(const __grid_constant__ Walk w, const __grid_constant__ DgArgs a) {
    __shared__ double sm[kDgThreads / 32];
    grid_wait();
    grid_next();
    const int Hv = w.p.Hv;
    const int32_t index = blockIdx.x / Hv;
    const int h = blockIdx.x % Hv, tid = threadIdx.x;
    const Part part = find_part(w, index, false);
    if (part.seq < 0 || part.t1 == part.t0) {
        if (a.part_sum && tid == 0) a.part_sum[(int64_t)index * Hv + h] = 0.0;
        return;
    }
    auto state = [&](const float* base, int64_t i) { return base ? base + (i * Hv + h) * (kD * kD) : nullptr; };
    double behind = part.last ? state_product(state(a.fin, part.seq), state(a.d_fin, part.seq), sm)
                              : state_product(state(w.joint, index + 1), state(a.joint_end, index), sm);
    const float* r = a.r + (int64_t)h * w.p.T;
    const float* c = a.c + (int64_t)h * w.p.T;
    double drift = 0.0;
    if (!part.first || !w.p.init || a.d_init) {
        double sum = 0.0;
        for (int64_t t = part.t0 + tid; t < part.t1; t += kDgThreads) sum += (double)r[t] - (double)c[t];
        sum = block_sum(sum, sm);
        const double front = part.first ? state_product(state(w.p.init, part.seq), state(a.d_init, part.seq), sm)
                                        : state_product(state(w.joint, index), state(a.joint_end, index - 1), sm);
        drift = (behind + sum - front) / (double)(part.t1 - part.t0);
        if (!(fabs(drift) <= 1e300)) drift = 0.0;          // a sequence with inf or NaN
    }
    double total = 0.0;
    for (int64_t end = part.t1; end > part.t0; end -= kDgThreads) {
        // thread 0 takes the last token of the block
        const int64_t t = end - 1 - tid;
        const bool there = t >= part.t0;
        double upto = there ? (double)r[t] - (double)c[t] : 0.0;
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const double y = __shfl_up_sync(0xffffffffu, upto, m);
            if ((tid & 31) >= m) upto += y;
        }
        if ((tid & 31) == 31) sm[tid >> 5] = upto;
        __syncthreads();
        double all = 0.0;
        for (int i = 0; i < kDgThreads / 32; ++i) {
            if (i < (tid >> 5)) upto += sm[i];
            all += sm[i];
        }
        __syncthreads();
        if (there) {
            const double d = w.p.g[t * w.p.ldg + h] <= kLinMinLogDecay
                                 ? 0.0 : behind + upto - drift * (double)(part.t1 - t);
            if (!a.part_sum) a.dg[t * Hv + h] = (float)d;
            total += d;
        }
        behind += all;
    }
    if (a.part_sum) {
        total = block_sum(total, sm);
        if (tid == 0) a.part_sum[(int64_t)index * Hv + h] = total;
    }
}

// dg of decays that all tokens share: the parts' sums, one warp per head
__global__ void lin_dg_sum_kernel(const double* part_sum, int32_t n_parts, int32_t Hv, float* dg) {
    const int h = blockIdx.x, lane = threadIdx.x;
    grid_wait();
    double s = 0.0;
    for (int i = lane; i < n_parts; i += 32) s += part_sum[(int64_t)i * Hv + h];
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
    if (lane == 0) dg[h] = (float)s;
}

// acc [tokens, width] in float32 -> out in bf16, for the tokens that sequences own; 8 elements a thread.  blockIdx.y:
// which of two.  Bound by HBM (8,192 tokens x 2,048: 16 us, half of what it reads still in L2)
struct Rounds {
    const float* acc[2];
    uint16_t* out[2];
};

__global__ void __launch_bounds__(256)
lin_round_kernel(const __grid_constant__ Rounds r, const int32_t* cu, int32_t n_seq, int64_t T, int32_t width) {
    grid_wait();
    grid_next();
    const float* acc = r.acc[blockIdx.y];
    uint16_t* out = r.out[blockIdx.y];
    const int64_t n = (cu ? (int64_t)cu[n_seq] : T) * (width / 8);
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
        const float4 a = reinterpret_cast<const float4*>(acc)[2 * i], b = reinterpret_cast<const float4*>(acc)[2 * i + 1];
        reinterpret_cast<uint4*>(out)[i] = make_uint4(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w),
                                                      pack_bf16x2(b.x, b.y), pack_bf16x2(b.z, b.w));
    }
}

// ---- launches -------------------------------------------------------------------------------------------
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// looked up once per process; null if the driver does not provide it
EncodeTiledFn encode_fn() {
    static const EncodeTiledFn fn = []() -> EncodeTiledFn {
        void* ptr = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &found) == cudaSuccess &&
            found == cudaDriverEntryPointSuccess)
            return reinterpret_cast<EncodeTiledFn>(ptr);
        cudaGetLastError();    // a refused query leaves no sticky error behind
        return nullptr;
    }();
    return fn;
}

// rows of an operand as 64 x 64 boxes, 128-byte swizzle
bool make_map(CUtensorMap* m, const LinOperand& o, int64_t T, int32_t Hv) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[2] = {(cuuint64_t)(Hv / o.rep) * kD, (cuuint64_t)T};
    cuuint64_t strides[1] = {(cuuint64_t)o.ld * 2};
    cuuint32_t box[2] = {64, 64};
    cuuint32_t estr[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<uint16_t*>(o.p), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// the output's rows as 32-row boxes of 128 bytes, 128-byte swizzle
bool make_out_map(CUtensorMap* m, const LinPass& p) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const bool f32 = p.out_rep > 1 || !p.out_bf16;
    void* base = f32 && p.out_bf16 ? p.acc : p.out;
    const cuuint64_t width = (cuuint64_t)(p.Hv / p.out_rep) * kD;
    cuuint64_t dims[2] = {width, (cuuint64_t)p.T};
    cuuint64_t strides[1] = {width * (f32 ? 4 : 2)};
    cuuint32_t box[2] = {f32 ? 32u : 64u, 32};
    cuuint32_t estr[2] = {1, 1};
    return fn(m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, base, dims, strides, box,
              estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// raises a kernel's limit of dynamic shared memory, once per device (`done`: the devices where it has been)
std::atomic<uint64_t> allowed[3][2];

cudaError_t allow_smem(const void* kernel, uint32_t bytes, std::atomic<uint64_t>& done) {
    int device = 0;
    cudaError_t e = cudaGetDevice(&device);
    if (e != cudaSuccess) return e;
    const uint64_t bit = device < 64 ? (uint64_t)1 << device : 0;
    if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

// kPasses passes that share their parts, heads and shape
template <int kMode, int kPasses>
cudaError_t launch_walk(const Walk* w, Chain& chain) {
    Passes<kPasses> ps{};
    for (int i = 0; i < kPasses; ++i) {
        const LinPass& p = w[i].p;
        if (!make_map(&ps.y[i], p.y, p.T, p.Hv) || !make_map(&ps.z[i], p.z, p.T, p.Hv) ||
            (kMode != kState && (!make_map(&ps.x[i], p.x, p.T, p.Hv) || !make_out_map(&ps.out[i], p))) ||
            (kMode == kExact && !make_map(&ps.u[i], p.u, p.T, p.Hv)))
            return cudaErrorInvalidValue;
        ps.w[i] = w[i];
    }
    ps.w[0].opens = !chain.begun;
    const LinPass& p = w[0].p;
    const int64_t blocks = kMode == kState ? (int64_t)w[0].n_inner * p.Hv : (int64_t)w[0].n_parts * (p.Hv / p.out_rep);
    if (blocks * kPasses > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    if (blocks == 0) return cudaSuccess;
    ps.blocks = (int32_t)blocks;
    const auto kernel = lin_walk_kernel<kMode, kPasses>;
    cudaError_t e = allow_smem(reinterpret_cast<const void*>(kernel), Layout<kMode>::kAlloc, allowed[kMode][kPasses - 1]);
    if (e != cudaSuccess) return e;
    e = chain.launch(true, kernel, (unsigned)(blocks * kPasses), kThreads, Layout<kMode>::kAlloc, ps);
    if (e != cudaSuccess) return e;
    if (kMode != kState && p.out_rep > 1 && p.out_bf16) {
        const int32_t width = p.Hv / p.out_rep * kD;
        const int64_t rows = (p.T * (width / 8) + 255) / 256;
        Rounds r{};
        for (int i = 0; i < kPasses; ++i) {
            r.acc[i] = w[i].p.acc;
            r.out[i] = static_cast<uint16_t*>(w[i].p.out);
        }
        e = chain.launch(true, lin_round_kernel, dim3((unsigned)(rows < kSms * 8 ? rows : kSms * 8), kPasses), 256, 0,
                         r, p.cu, p.n_seq, p.T, width);
    }
    return e;
}

// the starting states of all parts: each part's own sum, then the scan
template <int kPasses>
cudaError_t launch_joints(const WalkPair& w, Chain& chain) {
    cudaError_t e = launch_walk<kState, kPasses>(w.w, chain);
    if (e != cudaSuccess) return e;
    const LinPass& p = w.w[0].p;
    const int seqs = p.n_seq < kScanSeqs ? p.n_seq : kScanSeqs;
    return chain.launch(true, lin_scan_kernel,
                        dim3((unsigned)(seqs * p.Hv), kD * kD / (kScanThreads * 4), kPasses), kScanThreads, 0, w);
}

// no tokens at all: the states pass through
cudaError_t pass_state(const float* from, float* to, int32_t n_seq, int32_t Hv, cudaStream_t s) {
    if (!to || to == from) return cudaSuccess;
    const size_t bytes = (size_t)n_seq * Hv * kD * kD * 4;
    return from ? cudaMemcpyAsync(to, from, bytes, cudaMemcpyDeviceToDevice, s) : cudaMemsetAsync(to, 0, bytes, s);
}

struct Joints {
    int32_t part_len, n_parts, n_inner, split;
    size_t state_bytes, decay_bytes, list_bytes;
};

Joints joints_of(int32_t n_seq, int64_t T, int32_t Hv, int32_t part_len) {
    Joints j;
    j.part_len = part_len;
    j.n_parts = part_count(n_seq, T, j.part_len);
    j.n_inner = (int32_t)(T / j.part_len);      // parts that are not the last of their sequence are whole
    j.split = T > j.part_len;
    if (!j.split) j.n_parts = n_seq;
    j.state_bytes = j.split ? up256((size_t)j.n_parts * Hv * kD * kD * 4) : 0;
    j.decay_bytes = j.split ? up256((size_t)j.n_parts * Hv * 4) : 0;
    // (a CTA of the kernels finds its part among up to 32 sequences itself)
    j.list_bytes = j.split && n_seq > 32 ? up256(((size_t)j.n_parts + j.n_inner + n_seq + 1) * 4) : 0;
    return j;
}

// fills in w's parts, writing the lists where there are any
cudaError_t set_parts(Walk& w, const Joints& j, char* lists, Chain& chain) {
    w.part_len = j.part_len; w.n_parts = j.n_parts; w.n_inner = j.n_inner; w.split = j.split;
    if (j.list_bytes == 0) return cudaSuccess;
    int32_t* part_seq = reinterpret_cast<int32_t*>(lists);
    int32_t* inner = part_seq + j.n_parts;
    int32_t* seq_first = inner + j.n_inner;
    w.part_seq = part_seq;
    w.inner = inner;
    w.seq_first = seq_first;
    return chain.launch(false, lin_parts_kernel, 1, kListThreads, 0, w, part_seq, inner, seq_first);
}

// A call's plan follows from the workspace it is given: the fastest that fits, or the one that needs least.  What that
// one needs grows with T and n_seq, so a workspace for the largest of several calls serves all of them, which the
// fastest plans' sizes, taken call by call, would not let it.
constexpr int64_t kAnyLength = (int64_t)1 << 30;
constexpr size_t kAnySize = ~(size_t)0;

size_t prefill_bytes(const Joints& j) { return kWsHeaderBytes + j.state_bytes + j.decay_bytes + j.list_bytes; }

Joints prefill_plan(int32_t n_seq, int64_t T, int32_t Hv, size_t workspace_bytes) {
    const auto fits = [&](int32_t len) { return prefill_bytes(joints_of(n_seq, T, Hv, len)) <= workspace_bytes; };
    return joints_of(n_seq, T, Hv, choose_part_len(n_seq, T, Hv, 1, kAnyLength, fits));
}

struct BackwardPlan {
    Joints j;
    size_t qdq, kdk, acc, fin, sums, fwd, bwd, decay_f, decay_b, lists, bytes;
};

BackwardPlan backward_layout(int32_t n_seq, int64_t T, int32_t Hqk, int32_t Hv, int32_t part_len) {
    BackwardPlan b;
    b.j = joints_of(n_seq, T, Hv, part_len);
    size_t off = kWsHeaderBytes;
    auto take = [&](size_t bytes) { const size_t at = off; off += up256(bytes); return at; };
    b.qdq = take((size_t)T * Hv * 4);
    b.kdk = take((size_t)T * Hv * 4);
    b.acc = take(Hv > Hqk ? (size_t)T * Hqk * kD * 4 : 0);
    b.fin = take((size_t)n_seq * Hv * kD * kD * 4);
    b.sums = take((size_t)b.j.n_parts * Hv * 8);
    b.fwd = take(b.j.state_bytes);
    b.bwd = take(b.j.state_bytes);
    b.decay_f = take(b.j.decay_bytes);
    b.decay_b = take(b.j.decay_bytes);
    b.lists = take(b.j.list_bytes);
    b.bytes = off;
    return b;
}

BackwardPlan backward_plan(int32_t n_seq, int64_t T, int32_t Hqk, int32_t Hv, size_t workspace_bytes) {
    const auto fits = [&](int32_t len) { return backward_layout(n_seq, T, Hqk, Hv, len).bytes <= workspace_bytes; };
    // parts of at most 4096 tokens: the decays' gradient is a running sum along a part
    return backward_layout(n_seq, T, Hqk, Hv, choose_part_len(n_seq, T, Hqk, Hv / Hqk, 4096, fits));
}

}  // namespace

size_t linear_prefill_workspace_bytes(int32_t n_seq, int64_t T, int32_t Hv) {
    return prefill_bytes(prefill_plan(n_seq, T, Hv, kAnySize));
}
size_t linear_prefill_least_bytes(int32_t n_seq, int64_t T, int32_t Hv) {
    return prefill_bytes(prefill_plan(n_seq, T, Hv, 0));
}

cudaError_t launch_linear_prefill(const LinearArgs& a, cudaStream_t s) {
    char* ws = static_cast<char*>(a.workspace);
    if (a.T == 0) {
        const cudaError_t e = cudaMemsetAsync(ws, 0, kWsHeaderBytes, s);
        return e == cudaSuccess ? pass_state(a.initial_state, a.final_state, a.n_seq, a.Hv, s) : e;
    }
    const Joints j = prefill_plan(a.n_seq, a.T, a.Hv, a.workspace_bytes);
    Walk w{};
    w.joint = reinterpret_cast<float*>(ws + kWsHeaderBytes);
    w.joint_decay = reinterpret_cast<float*>(ws + kWsHeaderBytes + j.state_bytes);
    w.err = reinterpret_cast<uint32_t*>(ws + kWsErrorWordOffset);
    LinPass& p = w.p;
    p.x = {a.q, a.ldq, a.Hv / a.Hqk};
    p.y = {a.k, a.ldk, a.Hv / a.Hqk};
    p.z = {a.v, a.ldv, 1};
    p.g = a.g; p.ldg = a.ldg; p.cu = a.cu_seqlens; p.n_seq = a.n_seq; p.T = a.T; p.Hv = a.Hv; p.scale = a.scale;
    p.init = a.initial_state; p.fin = a.final_state;
    p.out = a.o; p.out_bf16 = a.o_bf16;
    Chain chain{s};
    cudaError_t e = set_parts(w, j, ws + kWsHeaderBytes + j.state_bytes + j.decay_bytes, chain);
    if (e != cudaSuccess) return e;
    if (j.split && (e = launch_joints<1>({{w}}, chain)) != cudaSuccess) return e;
    return launch_walk<kOut, 1>(&w, chain);
}

size_t linear_backward_workspace_bytes(int32_t n_seq, int64_t T, int32_t Hqk, int32_t Hv) {
    return backward_plan(n_seq, T, Hqk, Hv, kAnySize).bytes;
}
size_t linear_backward_least_bytes(int32_t n_seq, int64_t T, int32_t Hqk, int32_t Hv) {
    return backward_plan(n_seq, T, Hqk, Hv, 0).bytes;
}

cudaError_t launch_linear_backward(const LinearBackwardArgs& a, cudaStream_t s) {
    const BackwardPlan b = backward_plan(a.n_seq, a.T, a.Hqk, a.Hv, a.workspace_bytes);
    char* ws = static_cast<char*>(a.workspace);
    auto floats = [&](size_t at) { return reinterpret_cast<float*>(ws + at); };
    cudaError_t e;
    if (a.T == 0) {
        if ((e = cudaMemsetAsync(ws, 0, kWsHeaderBytes, s)) != cudaSuccess) return e;
        e = pass_state(a.d_final_state, a.d_initial_state, a.n_seq, a.Hv, s);
        return e == cudaSuccess && !a.ldg ? cudaMemsetAsync(a.dg, 0, (size_t)a.Hv * 4, s) : e;
    }
    const int rep = a.Hv / a.Hqk;
    const LinOperand q{a.q, a.ldq, rep}, k{a.k, a.ldk, rep}, v{a.v, a.ldv, 1}, d_o{a.d_o, (int64_t)a.Hv * kD, 1};
    Walk base{};
    base.err = reinterpret_cast<uint32_t*>(ws + kWsErrorWordOffset);
    base.p.g = a.g; base.p.ldg = a.ldg; base.p.cu = a.cu_seqlens; base.p.n_seq = a.n_seq; base.p.T = a.T;
    base.p.Hv = a.Hv; base.p.scale = a.scale; base.p.out_bf16 = a.grad_bf16;
    Chain chain{s};
    if ((e = set_parts(base, b.j, ws + b.lists, chain)) != cudaSuccess) return e;
    Walk fwd = base, bwd = base;
    fwd.joint = floats(b.fwd); fwd.joint_decay = floats(b.decay_f);
    bwd.joint = floats(b.bwd); bwd.joint_decay = floats(b.decay_b);
    bwd.p.backward = 1;
    if (b.j.split) {                            // S at the parts' starts, dS at their ends
        WalkPair w{{fwd, bwd}};
        w.w[0].p.y = k; w.w[0].p.z = v; w.w[0].p.init = a.initial_state;
        w.w[1].p.y = q; w.w[1].p.z = d_o; w.w[1].p.init = a.d_final_state;
        if ((e = launch_joints<2>(w, chain)) != cudaSuccess) return e;
    }
    float* fin = a.d_final_state ? floats(b.fin) : nullptr;
    Walk both[2] = {fwd, bwd};
    LinPass& dq = both[0].p;                    // its state is S^T
    dq.x = d_o; dq.y = v; dq.z = k; dq.u = q; dq.dots = floats(b.qdq);
    dq.init = a.initial_state; dq.fin = fin; dq.state_t = 1; both[0].joint_t = 1;
    dq.out = a.dq; dq.out_rep = rep; dq.acc = floats(b.acc);
    LinPass& dk = both[1].p;                    // dS^T
    dk.x = v; dk.y = d_o; dk.z = q; dk.u = k; dk.dots = floats(b.kdk);
    dk.init = a.d_final_state; dk.state_t = 1; both[1].joint_t = 1;
    dk.out = a.dk; dk.out_rep = rep;
    // Where both fill no more than one round of CTAs, they share it (572 ragged tokens, 24 CTAs each: 100 -> 81 us for
    // the whole backward), and dk's rows are summed where dv's will be written (as large at least: rep > 1).  Beyond
    // that they take turns, with one accumulator and the faster kernel for one pass (8,192 tokens, 144 CTAs each: in one
    // launch the whole backward took 735 us for 650).
    const bool pair = 2 * (int64_t)b.j.n_parts * a.Hqk <= kSms;
    dk.acc = pair ? static_cast<float*>(a.dv) : floats(b.acc);
    if (pair) {
        if ((e = launch_walk<kExact, 2>(both, chain)) != cudaSuccess) return e;
    } else if ((e = launch_walk<kExact, 1>(both, chain)) != cudaSuccess ||
               (e = launch_walk<kExact, 1>(both + 1, chain)) != cudaSuccess) {
        return e;
    }
    Walk w = bwd;                               // dv: dS
    w.p.x = k; w.p.y = q; w.p.z = d_o;
    w.p.init = a.d_final_state; w.p.fin = a.d_initial_state;
    w.p.out = a.dv;
    if ((e = launch_walk<kOut, 1>(&w, chain)) != cudaSuccess) return e;
    double* sums = a.ldg ? nullptr : reinterpret_cast<double*>(ws + b.sums);
    fwd.p.init = a.initial_state;
    const DgArgs dg{floats(b.qdq), floats(b.kdk), bwd.joint, fin, a.d_final_state, a.d_initial_state, a.dg, sums};
    // (not ahead of time: its CTAs, eight to an SM, then crowd the SMs that fall free first, 670 us for 655 at 8,192
    // tokens)
    e = chain.launch(false, lin_dg_kernel, (unsigned)(b.j.n_parts * a.Hv), kDgThreads, 0, fwd, dg);
    if (e != cudaSuccess || a.ldg) return e;
    return chain.launch(false, lin_dg_sum_kernel, a.Hv, 32, 0, sums, b.j.n_parts, a.Hv, a.dg);
}

}  // namespace gdn
