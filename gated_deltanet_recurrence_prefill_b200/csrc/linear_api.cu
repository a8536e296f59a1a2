// linear_api.cu -- the C ABI of the linear attention with a decay per head and of
// the state cache's pages (include/gdn.h): argument checks on the host, then
// kernel launches on the caller's stream.
#include <cuda_runtime.h>

#include "../../include/gdn.h"
#include "kernels.h"

namespace {

constexpr int32_t kD = 128;
constexpr int32_t kMostSlots = 1 << 24;           // of a cache, and entries of a list

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

gdn_status done(cudaError_t e) { return e == cudaSuccess ? GDN_OK : gdn::set_last_cuda_error(e); }

bool flag(int32_t x) { return x == 0 || x == 1; }

gdn_status check_heads(int32_t Hqk, int32_t Hv, int32_t d) {
    if (Hqk <= 0 || Hv <= 0 || d <= 0) return GDN_ERR_INVALID_ARG;
    if (d != kD || Hv % Hqk != 0 || Hv > 65535) return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}

gdn_status check_seqs(const int32_t* cu_seqlens, int32_t n_seq, int64_t T, int32_t Hv) {
    if (T < 0 || n_seq <= 0) return GDN_ERR_INVALID_ARG;
    if (!cu_seqlens && n_seq != 1) return GDN_ERR_INVALID_ARG;
    if (T > (int64_t)0x7fffff00) return GDN_ERR_UNSUPPORTED;                  // cu_seqlens are int32
    if ((int64_t)n_seq * Hv > (int64_t)0x3fffffff) return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}

// the elements from a token to the next: 0 stands for the dense heads * d
gdn_status check_ld(int64_t& ld, int32_t heads) {
    if (ld == 0) ld = (int64_t)heads * kD;
    if (ld < (int64_t)heads * kD) return GDN_ERR_INVALID_ARG;
    if (ld % 8 != 0) return GDN_ERR_MISALIGNED;
    if (ld > ((int64_t)1 << 38)) return GDN_ERR_UNSUPPORTED;                 // a tensor map's strides are below 2^40 bytes
    return GDN_OK;
}

gdn_status check_workspace(const void* workspace, size_t bytes, size_t need, uintptr_t align) {
    if (!workspace || bytes < need) return GDN_ERR_WORKSPACE;
    return aligned(workspace, align) ? GDN_OK : GDN_ERR_MISALIGNED;
}

gdn_status check_buffers(const gdn_state_buffer* buffers, int32_t n_buffers, int32_t n_slots, gdn::StateBuffers& b) {
    static_assert(GDN_MAX_STATE_BUFFERS == gdn::kMaxStateBuffers && GDN_MAX_STATE_COPIES == gdn::kMaxStateCopies,
                  "the header's limits");
    if (n_buffers < 0 || n_slots <= 0 || (n_buffers > 0 && !buffers)) return GDN_ERR_INVALID_ARG;
    if (n_buffers > GDN_MAX_STATE_BUFFERS || n_slots > kMostSlots) return GDN_ERR_UNSUPPORTED;
    for (int i = 0; i < n_buffers; ++i) {
        if (!buffers[i].data || buffers[i].slot_bytes <= 0) return GDN_ERR_INVALID_ARG;
        if (!aligned(buffers[i].data, 16) || buffers[i].slot_bytes % 16 != 0) return GDN_ERR_MISALIGNED;
        if (buffers[i].slot_bytes > ((int64_t)1 << 38)) return GDN_ERR_UNSUPPORTED;
        b.data[i] = static_cast<uint8_t*>(buffers[i].data);
        b.bytes[i] = buffers[i].slot_bytes;
        for (int k = 0; k < i; ++k)            // a buffer named twice would be moved twice
            if (b.data[k] < b.data[i] + b.bytes[i] * n_slots && b.data[i] < b.data[k] + b.bytes[k] * n_slots)
                return GDN_ERR_INVALID_ARG;
    }
    b.n = n_buffers;
    b.n_slots = n_slots;
    return GDN_OK;
}

}  // namespace

extern "C" {

size_t gdn_linear_prefill_workspace_size(int32_t n_seq, int64_t T, int32_t Hqk, int32_t Hv, int32_t d) {
    (void)Hqk; (void)d;
    return gdn::linear_prefill_workspace_bytes(n_seq > 0 ? n_seq : 1, T > 0 ? T : 0, Hv > 0 ? Hv : 1);
}

gdn_status gdn_linear_prefill(const uint16_t* q, const uint16_t* k, const uint16_t* v, int64_t ldq, int64_t ldk,
                              int64_t ldv, const float* g, int32_t g_per_token, const int32_t* cu_seqlens,
                              int32_t n_seq, int64_t T, int32_t Hqk, int32_t Hv, int32_t d, float scale,
                              const float* initial_state, float* final_state, void* o, int32_t o_bf16,
                              void* workspace, size_t workspace_bytes, gdn_stream_t stream) {
    gdn_status st = check_heads(Hqk, Hv, d);
    if (st != GDN_OK) return st;
    if ((st = check_seqs(cu_seqlens, n_seq, T, Hv)) != GDN_OK) return st;
    if (!flag(g_per_token) || !flag(o_bf16)) return GDN_ERR_INVALID_ARG;
    if (T > 0 && (!q || !k || !v || !g || !o)) return GDN_ERR_INVALID_ARG;
    if ((st = check_ld(ldq, Hqk)) != GDN_OK || (st = check_ld(ldk, Hqk)) != GDN_OK || (st = check_ld(ldv, Hv)) != GDN_OK)
        return st;
    const void* ptrs[] = {q, k, v, g, cu_seqlens, initial_state, final_state, o};
    for (const void* p : ptrs)
        if (!aligned(p, 16)) return GDN_ERR_MISALIGNED;
    st = check_workspace(workspace, workspace_bytes, gdn::linear_prefill_least_bytes(n_seq, T, Hv), 256);
    if (st != GDN_OK) return st;
    gdn::LinearArgs a{q, k, v, ldq, ldk, ldv, g, g_per_token ? Hv : 0, cu_seqlens, n_seq, T, Hqk, Hv, scale,
                      initial_state, final_state, o, o_bf16, workspace, workspace_bytes};
    return done(gdn::launch_linear_prefill(a, (cudaStream_t)stream));
}

size_t gdn_linear_prefill_backward_workspace_size(int32_t n_seq, int64_t T, int32_t Hqk, int32_t Hv, int32_t d) {
    (void)d;
    return gdn::linear_backward_workspace_bytes(n_seq > 0 ? n_seq : 1, T > 0 ? T : 0, Hqk > 0 ? Hqk : 1,
                                                Hv > 0 ? Hv : 1);
}

gdn_status gdn_linear_prefill_backward(const uint16_t* q, const uint16_t* k, const uint16_t* v, int64_t ldq,
                                       int64_t ldk, int64_t ldv, const float* g, int32_t g_per_token,
                                       const int32_t* cu_seqlens, int32_t n_seq, int64_t T, int32_t Hqk, int32_t Hv,
                                       int32_t d, float scale, const float* initial_state, const uint16_t* d_o,
                                       const float* d_final_state, void* dq, void* dk, void* dv, int32_t grad_bf16,
                                       float* dg, float* d_initial_state, void* workspace, size_t workspace_bytes,
                                       gdn_stream_t stream) {
    gdn_status st = check_heads(Hqk, Hv, d);
    if (st != GDN_OK) return st;
    if ((st = check_seqs(cu_seqlens, n_seq, T, Hv)) != GDN_OK) return st;
    if (!flag(g_per_token) || !flag(grad_bf16)) return GDN_ERR_INVALID_ARG;
    if (!g_per_token && !dg) return GDN_ERR_INVALID_ARG;
    if (T > 0 && (!q || !k || !v || !g || !d_o || !dq || !dk || !dv || !dg)) return GDN_ERR_INVALID_ARG;
    if (d_initial_state && (d_initial_state == d_final_state || d_initial_state == initial_state))
        return GDN_ERR_INVALID_ARG;
    if ((st = check_ld(ldq, Hqk)) != GDN_OK || (st = check_ld(ldk, Hqk)) != GDN_OK || (st = check_ld(ldv, Hv)) != GDN_OK)
        return st;
    const void* ptrs[] = {q, k, v, g, cu_seqlens, initial_state, d_o, d_final_state, dq, dk, dv, dg, d_initial_state};
    for (const void* p : ptrs)
        if (!aligned(p, 16)) return GDN_ERR_MISALIGNED;
    st = check_workspace(workspace, workspace_bytes, gdn::linear_backward_least_bytes(n_seq, T, Hqk, Hv), 256);
    if (st != GDN_OK) return st;
    gdn::LinearBackwardArgs a{q, k, v, ldq, ldk, ldv, g, g_per_token ? Hv : 0, cu_seqlens, n_seq, T, Hqk, Hv, scale,
                              initial_state, d_o, d_final_state, dq, dk, dv, grad_bf16, dg, d_initial_state,
                              workspace, workspace_bytes};
    return done(gdn::launch_linear_backward(a, (cudaStream_t)stream));
}

gdn_status gdn_linear_decode_step(const uint16_t* q, const uint16_t* k, const uint16_t* v, const float* g,
                                  int32_t g_per_unit, const int32_t* slot, int32_t n_seq, int32_t layers, int32_t Hqk,
                                  int32_t Hv, int32_t d, float scale, int32_t n_slots, void* state,
                                  int32_t state_bf16, void* o, int32_t o_bf16, gdn_stream_t stream) {
    gdn_status st = check_heads(Hqk, Hv, d);
    if (st != GDN_OK) return st;
    if (n_seq < 0 || layers <= 0 || n_slots < 0 || !flag(g_per_unit) || !flag(state_bf16) || !flag(o_bf16))
        return GDN_ERR_INVALID_ARG;
    if (!slot && n_slots < n_seq) return GDN_ERR_INVALID_ARG;
    if (n_seq == 0) return GDN_OK;
    if (!q || !k || !v || !g || !o || (n_slots > 0 && !state)) return GDN_ERR_INVALID_ARG;
    if ((int64_t)n_seq * layers > 0x7fffffffLL / Hv) return GDN_ERR_UNSUPPORTED;
    const void* ptrs[] = {q, k, v, g, slot, state, o};
    for (const void* p : ptrs)
        if (!aligned(p, 16)) return GDN_ERR_MISALIGNED;
    gdn::LinearDecodeArgs a{q, k, v, g, g_per_unit, slot, n_seq, layers, Hqk, Hv, scale, n_slots, state, state_bf16,
                            o, o_bf16};
    return done(gdn::launch_linear_decode(a, (cudaStream_t)stream));
}

gdn_status gdn_state_copy(const gdn_state_buffer* buffers, int32_t n_buffers, int32_t n_slots, const int32_t* src,
                          const int32_t* dst, int32_t n, gdn_stream_t stream) {
    gdn::StateBuffers b;
    gdn_status st = check_buffers(buffers, n_buffers, n_slots, b);
    if (st != GDN_OK) return st;
    if (n < 0) return GDN_ERR_INVALID_ARG;
    if (n > GDN_MAX_STATE_COPIES) return GDN_ERR_UNSUPPORTED;
    if (n == 0 || n_buffers == 0) return GDN_OK;
    if (!src || !dst) return GDN_ERR_INVALID_ARG;
    if (!aligned(src, 4) || !aligned(dst, 4)) return GDN_ERR_MISALIGNED;
    return done(gdn::launch_state_copy(b, src, dst, n, (cudaStream_t)stream));
}

size_t gdn_state_workspace_size(int32_t n_slots) { return gdn::state_workspace_bytes(n_slots > 0 ? n_slots : 1); }

gdn_status gdn_state_fork(const gdn_state_buffer* buffers, int32_t n_buffers, int32_t n_slots, int32_t* live,
                          const int32_t* src, int32_t* dst, int32_t n, void* workspace, size_t workspace_bytes,
                          gdn_stream_t stream) {
    gdn::StateBuffers b;
    gdn_status st = check_buffers(buffers, n_buffers, n_slots, b);
    if (st != GDN_OK) return st;
    if (n < 0 || !live) return GDN_ERR_INVALID_ARG;
    if (n > kMostSlots) return GDN_ERR_UNSUPPORTED;
    if (n == 0) return GDN_OK;
    if (!src || !dst || src == dst || dst == live) return GDN_ERR_INVALID_ARG;
    if (!aligned(src, 4) || !aligned(dst, 4) || !aligned(live, 4)) return GDN_ERR_MISALIGNED;
    if ((st = check_workspace(workspace, workspace_bytes, gdn::state_workspace_bytes(n_slots), 16)) != GDN_OK) return st;
    return done(gdn::launch_state_fork(b, live, src, dst, n, workspace, (cudaStream_t)stream));
}

gdn_status gdn_state_compact(const gdn_state_buffer* buffers, int32_t n_buffers, int32_t n_slots, int32_t* live,
                             int32_t* moved, void* workspace, size_t workspace_bytes, gdn_stream_t stream) {
    gdn::StateBuffers b;
    gdn_status st = check_buffers(buffers, n_buffers, n_slots, b);
    if (st != GDN_OK) return st;
    if (!live || !moved || live == moved) return GDN_ERR_INVALID_ARG;
    if (!aligned(moved, 4) || !aligned(live, 4)) return GDN_ERR_MISALIGNED;
    if ((st = check_workspace(workspace, workspace_bytes, gdn::state_workspace_bytes(n_slots), 16)) != GDN_OK) return st;
    return done(gdn::launch_state_compact(b, live, moved, workspace, (cudaStream_t)stream));
}

gdn_status gdn_state_free(int32_t* live, int32_t n_slots, const int32_t* slots, int32_t n, gdn_stream_t stream) {
    if (n_slots <= 0 || n < 0 || !live) return GDN_ERR_INVALID_ARG;
    if (n_slots > kMostSlots || n > kMostSlots) return GDN_ERR_UNSUPPORTED;
    if (n == 0) return GDN_OK;
    if (!slots) return GDN_ERR_INVALID_ARG;
    if (!aligned(slots, 4) || !aligned(live, 4)) return GDN_ERR_MISALIGNED;
    return done(gdn::launch_state_free(live, n_slots, slots, n, (cudaStream_t)stream));
}

}  // extern "C"
