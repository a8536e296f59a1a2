// linear_token.cu -- the linear attention passes of linear_attn.h one token at a
// time in float32 on the CUDA cores.  One CTA of 128 threads per (sequence,
// output head): thread i holds row i of the state in registers, the token's x
// and y rows go through shared memory, and the value heads that share an output
// row are taken in turn.
#include "common.cuh"
#include "kernels.h"
#include "linear_attn.h"

namespace gdn {

namespace {

constexpr int kD = 128;

GDN_DEVICE float operand(const LinOperand& o, int64_t t, int h, int i) {
    return bf16_to_f32(o.p[t * o.ld + (int64_t)(h / o.rep) * kD + i]);
}

__global__ void __launch_bounds__(kD) lin_token_kernel(LinPass p) {
    __shared__ __align__(16) float xs[kD], ys[kD];
    __shared__ float part[4];
    const int i = threadIdx.x;
    const int heads = p.Hv / p.out_rep;
    const int seq = blockIdx.x / heads, ho = blockIdx.x % heads;
    const int64_t t0 = p.cu ? p.cu[seq] : 0, t1 = p.cu ? p.cu[seq + 1] : p.T;
    for (int j = 0; j < p.out_rep; ++j) {
        const int h = ho * p.out_rep + j;
        const int64_t sbase = ((int64_t)seq * p.Hv + h) * kD * kD;
        const int64_t rs = p.state_t ? 1 : kD, cs = p.state_t ? kD : 1;
        float A[kD];
#pragma unroll
        for (int c = 0; c < kD; ++c) A[c] = p.init ? p.init[sbase + i * rs + c * cs] : 0.f;
        for (int64_t n = 0; n < t1 - t0; ++n) {
            const int64_t t = p.backward ? t1 - 1 - n : t0 + n;
            float g = p.g[t * p.ldg + h];
            g = g < kLinMinLogDecay ? kLinMinLogDecay : g;
            const float decay = expf(g);
            xs[i] = operand(p.x, t, h, i);
            ys[i] = operand(p.y, t, h, i);
            const float z = operand(p.z, t, h, i) * (p.backward ? p.scale : 1.f);
            __syncthreads();
            float o = 0.f;
            const float before = p.backward ? 1.f : decay, behind = p.backward ? decay : 1.f;
#pragma unroll
            for (int c = 0; c < kD; ++c) {
                const float s = fmaf(before, A[c], z * ys[c]);
                o = fmaf(s, xs[c], o);
                A[c] = behind * s;
            }
            if (!p.backward) o *= p.scale;
            if (p.dots) {
                const float w = warp_sum(o * operand(p.u, t, h, i));
                if ((i & 31) == 0) part[i >> 5] = w;
            }
            const int64_t at = (t * heads + ho) * kD + i;
            float sum = o;
            float* acc = p.out_rep == 1 ? nullptr : p.out_bf16 ? p.acc : static_cast<float*>(p.out);
            if (j > 0) sum += acc[at];
            if (j + 1 < p.out_rep)
                acc[at] = sum;
            else if (p.out_bf16)
                static_cast<uint16_t*>(p.out)[at] = (uint16_t)f32_to_bf16_bits(sum);
            else
                static_cast<float*>(p.out)[at] = sum;
            __syncthreads();
            if (p.dots && i == 0) p.dots[t * p.Hv + h] = (part[0] + part[1]) + (part[2] + part[3]);
        }
        if (p.fin)
#pragma unroll
            for (int c = 0; c < kD; ++c) p.fin[sbase + i * rs + c * cs] = A[c];
    }
}

// the decays' gradient from the two dot products per token (linear_attn.h's
// passes): with B_t = <S_t, dS_t>, dS_t the whole gradient at S_t,
//   B_t gains q_t . dq_t,  dg_t = B_t - k_t . dk_t,  B_{t-1} = dg_t,
// from the last token back, B starting at <S_T, dL/dS_T>.  One warp per
// (sequence, head), the sum in 64 bits.
__global__ void lin_dg_token_kernel(const float* qdq, const float* kdk, const float* g, int64_t ldg,
                                    const int32_t* cu, int64_t T, int32_t n_seq, int32_t Hv, const float* fin,
                                    const float* d_fin, float* dg, double* per_seq) {
    const int lane = threadIdx.x;
    const int seq = blockIdx.x / Hv, h = blockIdx.x % Hv;
    const int64_t t0 = cu ? cu[seq] : 0, t1 = cu ? cu[seq + 1] : T;
    double B = 0.0;
    if (d_fin) {
        const int64_t base = ((int64_t)seq * Hv + h) * kD * kD;
        for (int i = lane; i < kD * kD; i += 32) B += (double)fin[base + i] * d_fin[base + i];
#pragma unroll
        for (int m = 16; m >= 1; m >>= 1) B += __shfl_xor_sync(0xffffffffu, B, m);
    }
    if (lane != 0) return;
    double total = 0.0;
    for (int64_t t = t1 - 1; t >= t0; --t) {
        B += (double)qdq[t * Hv + h] - (double)kdk[t * Hv + h];
        const double d = g[t * ldg + h] <= kLinMinLogDecay ? 0.0 : B;
        if (ldg) dg[t * Hv + h] = (float)d;
        total += d;
    }
    if (!ldg) per_seq[(int64_t)seq * Hv + h] = total;
}

__global__ void lin_dg_sum_kernel(const double* per_seq, int32_t n_seq, int32_t Hv, float* dg) {
    const int h = blockIdx.x * blockDim.x + threadIdx.x;
    if (h >= Hv) return;
    double s = 0.0;
    for (int i = 0; i < n_seq; ++i) s += per_seq[(int64_t)i * Hv + h];
    dg[h] = (float)s;
}

size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

struct BackwardPlan {
    size_t qdq, kdk, acc, fin, sums, bytes;
};

BackwardPlan backward_plan(int32_t n_seq, int64_t T, int32_t Hqk, int32_t Hv) {
    BackwardPlan b;
    size_t off = kWsHeaderBytes;
    b.qdq = off; off += up256((size_t)T * Hv * 4);
    b.kdk = off; off += up256((size_t)T * Hv * 4);
    b.acc = off; off += up256((size_t)T * Hqk * kD * 4);
    b.fin = off; off += up256((size_t)n_seq * Hv * kD * kD * 4);
    b.sums = off; off += up256((size_t)n_seq * Hv * 8);
    b.bytes = off;
    return b;
}

cudaError_t run_pass(const LinPass& p, cudaStream_t s) {
    const int64_t blocks = (int64_t)p.n_seq * (p.Hv / p.out_rep);
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    lin_token_kernel<<<(unsigned)blocks, kD, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace

size_t linear_prefill_workspace_bytes(int32_t n_seq, int64_t T, int32_t Hv) {
    (void)n_seq; (void)T; (void)Hv;
    return kWsHeaderBytes;
}

cudaError_t launch_linear_prefill(const LinearArgs& a, cudaStream_t s) {
    LinPass p;
    p.x = {a.q, a.ldq, a.Hv / a.Hqk};
    p.y = {a.k, a.ldk, a.Hv / a.Hqk};
    p.z = {a.v, a.ldv, 1};
    p.g = a.g; p.ldg = a.ldg; p.cu = a.cu_seqlens; p.n_seq = a.n_seq; p.T = a.T; p.Hv = a.Hv; p.scale = a.scale;
    p.init = a.initial_state; p.fin = a.final_state;
    p.out = a.o; p.out_bf16 = a.o_bf16;
    cudaError_t e = cudaMemsetAsync(a.workspace, 0, kWsHeaderBytes, s);
    return e == cudaSuccess ? run_pass(p, s) : e;
}

size_t linear_backward_workspace_bytes(int32_t n_seq, int64_t T, int32_t Hqk, int32_t Hv) {
    return backward_plan(n_seq, T, Hqk, Hv).bytes;
}

cudaError_t launch_linear_backward(const LinearBackwardArgs& a, cudaStream_t s) {
    const BackwardPlan b = backward_plan(a.n_seq, a.T, a.Hqk, a.Hv);
    char* ws = static_cast<char*>(a.workspace);
    const int rep = a.Hv / a.Hqk;
    const LinOperand q{a.q, a.ldq, rep}, k{a.k, a.ldk, rep}, v{a.v, a.ldv, 1}, d_o{a.d_o, (int64_t)a.Hv * kD, 1};
    LinPass base;
    base.g = a.g; base.ldg = a.ldg; base.cu = a.cu_seqlens; base.n_seq = a.n_seq; base.T = a.T; base.Hv = a.Hv;
    base.scale = a.scale; base.out_bf16 = a.grad_bf16;
    float* fin = a.d_final_state ? reinterpret_cast<float*>(ws + b.fin) : nullptr;
    float* acc = reinterpret_cast<float*>(ws + b.acc);
    LinPass p = base;                           // dq
    p.x = d_o; p.y = v; p.z = k; p.u = q; p.dots = reinterpret_cast<float*>(ws + b.qdq);
    p.init = a.initial_state; p.fin = fin; p.state_t = 1;
    p.out = a.dq; p.out_rep = rep; p.acc = acc;
    cudaError_t e = cudaMemsetAsync(a.workspace, 0, kWsHeaderBytes, s);
    if (e == cudaSuccess) e = run_pass(p, s);
    if (e != cudaSuccess) return e;
    p = base;                                   // dk
    p.backward = 1;
    p.x = v; p.y = d_o; p.z = q; p.u = k; p.dots = reinterpret_cast<float*>(ws + b.kdk);
    p.init = a.d_final_state; p.state_t = 1;
    p.out = a.dk; p.out_rep = rep; p.acc = acc;
    if ((e = run_pass(p, s)) != cudaSuccess) return e;
    p = base;                                   // dv
    p.backward = 1;
    p.x = k; p.y = q; p.z = d_o;
    p.init = a.d_final_state; p.fin = a.d_initial_state;
    p.out = a.dv;
    if ((e = run_pass(p, s)) != cudaSuccess) return e;
    double* sums = reinterpret_cast<double*>(ws + b.sums);
    lin_dg_token_kernel<<<(unsigned)(a.n_seq * a.Hv), 32, 0, s>>>(
        reinterpret_cast<float*>(ws + b.qdq), reinterpret_cast<float*>(ws + b.kdk), a.g, a.ldg, a.cu_seqlens, a.T,
        a.n_seq, a.Hv, fin, a.d_final_state, a.dg, sums);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    if (!a.ldg) {
        lin_dg_sum_kernel<<<(a.Hv + 127) / 128, 128, 0, s>>>(sums, a.n_seq, a.Hv, a.dg);
        e = cudaGetLastError();
    }
    return e;
}

}  // namespace gdn
