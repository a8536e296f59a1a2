// linear_attn.h -- internal interface of the linear attention with a decay per
// head (gdn_linear_*): one pass over packed sequences, in either direction.
//
// Per value head, with A (128 x 128, rows the z index, columns the y index),
//   forward    A <- e^{g_t} A + z_t y_t^T,           out_t = scale A x_t
//   backward   A <- A + scale z_t y_t^T, out_t = A x_t, A <- e^{g_t} A   (t falling)
// The prefill is the forward pass with (x, y, z) = (q, k, v).  Its gradients are
//   dq: forward  with (d_o, v, k)   (the state is S^T)
//   dk: backward with (v, d_o, q)   (the state is dS^T)
//   dv: backward with (k, q, d_o)   (the state is dS)
// because o_t = scale sum_{s<=t} e^{G_t - G_s} (q_t . k_s) v_s + scale e^{G_t} S_0 q_t is
// linear in each of q, k and v, and S enters the loss through the same sums.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace gdn {

// bf16 rows of 128 per (token, head): row (t, h) at p + t * ld + (h / rep) * 128
struct LinOperand {
    const uint16_t* p = nullptr;
    int64_t ld = 0;
    int32_t rep = 1;
};

struct LinPass {
    LinOperand x, y, z;
    LinOperand u;                       // dots[t, h] = u_t . out_t (float32) when dots is given
    float* dots = nullptr;              // [Hv, T]
    const float* g = nullptr;           // log decays: row t at g + t * ldg (ldg = 0: one per head)
    int64_t ldg = 0;
    const int32_t* cu = nullptr;        // NULL: one sequence of length T
    int32_t n_seq = 1;
    int64_t T = 0;
    int32_t Hv = 0;
    float scale = 1.f;
    int32_t backward = 0;
    // the state at the pass's start and end ([n_seq, Hv, 128, 128] or NULL), stored transposed
    // (columns the z index) when state_t is set
    const float* init = nullptr;
    float* fin = nullptr;
    int32_t state_t = 0;
    // out: row (t, h) at (t * Hv / out_rep + h / out_rep) * 128, the out_rep value heads that share a
    // row summed in float32 (through acc [T, Hv / out_rep, 128] when out_rep > 1 and out is bf16)
    void* out = nullptr;
    int32_t out_bf16 = 0;
    int32_t out_rep = 1;
    float* acc = nullptr;
};

// log decays below this are taken as this: e^-104 is 0 in float32, so a log decay of -inf (a reset)
// stays finite in sums and differences; NaN stays NaN
constexpr float kLinMinLogDecay = -104.f;

}  // namespace gdn
