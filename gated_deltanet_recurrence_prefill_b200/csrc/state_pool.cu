// state_pool.cu -- pages of a state cache: copying, forking, compacting, freeing.
//
// A cache is up to kMaxStateBuffers arrays whose leading axis is the slot (the
// recurrent states, the convolution histories, ...); a page is one slot of all
// of them.  Everything here moves bytes, bound by HBM bandwidth; a page of a
// whole model is tens of megabytes, so the lists are worked out by small
// kernels whose time does not show, and the moves run on every SM.
#include "common.cuh"
#include "kernels.h"
#include "launch_chain.h"

namespace gdn {

namespace {

GDN_DEVICE uint32_t smem_addr(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }

GDN_DEVICE void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// ---- copy: page[dst[i]] = (old page)[src[i]], all entries at once ----------------------------------
//
// Any entry may read a page that another one overwrites (a reordering in place).
// A work item is one range of bytes of a page, taken for every entry: the CTA
// brings the range of all sources into shared memory and then writes it to all
// destinations, so every read of the range comes before every write of it, and
// no two items touch the same bytes.  No second cache and no order of moves is
// needed; a page is written once, and loaded for every entry that reads it (from L2
// after the first).  Bound by HBM, whose rate falls where reads and writes of short
// ranges take turns: 57 pages of 77 MB (with their conv histories) from 23, 6.3 GB
// to move, in 1.14 ms one call after another (5.5 TB/s; 1.24 ms by itself) with
// ranges of 1,792 bytes; with half the room, 512 bytes and two CTAs an SM 4.9 TB/s,
// with one item at a time 4.4.  384 threads: 512 took 1.16 ms, 640 1.17.  Pages of
// their own, 16 MB from 256: 5.1 TB/s, 4 MB from 832 (128 bytes) 4.3, from more
// (64 bytes) 2.3.
constexpr int kCopyThreads = 384;
constexpr int kCopyStage = 104 * 1024;         // bytes of an item; a CTA has room for two, an SM for one CTA
constexpr int kCopyMostRange = 32 * 1024, kCopyStep = 128, kCopyMinRange = 64;      // bytes of a page in an item
constexpr int kCopyMostSmem = 2 * kCopyStage + 8 * (kCopyStage / kCopyStep);
static_assert(kCopyMostSmem >= kMaxStateCopies * (2 * kCopyMinRange + 8) && kCopyMostSmem <= 227 * 1024,
              "the most that any number of entries takes");

__global__ void __launch_bounds__(kCopyThreads, 1)
state_copy_kernel(StateBuffers b, const int32_t* __restrict__ src, const int32_t* __restrict__ dst, int32_t n,
                  int32_t range) {
    extern __shared__ __align__(16) uint8_t sm[];
    uint8_t* stage = sm;
    int32_t* from = reinterpret_cast<int32_t*>(sm + 2 * (size_t)n * range);
    int32_t* to = from + n;
    __shared__ int32_t count;
    const int tid = threadIdx.x;
    if (tid == 0) count = 0;
    for (int i = tid; i < n; i += kCopyThreads) {
        const int32_t s = src[i], d = dst[i];
        const bool there = s >= 0 && s < b.n_slots && d >= 0 && d < b.n_slots;      // else the entry is ignored
        to[i] = there ? d : -1;
    }
    __syncthreads();
    // the entries that move something: of several with one destination the last
    for (int i = tid; i < n; i += kCopyThreads) {
        const int32_t s = src[i], d = to[i];
        bool keep = d >= 0 && s != d;
        for (int j = i + 1; keep && j < n; ++j) keep = to[j] != d;
        from[i] = keep ? s : -1;
    }
    __syncthreads();
    // closed up, in order, by one warp
    if (tid < 32) {
        int at = 0;
        for (int i0 = 0; i0 < n; i0 += 32) {
            const int i = i0 + tid;
            const int32_t s = i < n ? from[i] : -1, d = i < n ? to[i] : -1;
            const unsigned m = __ballot_sync(0xffffffffu, s >= 0);
            __syncwarp();
            if (s >= 0) {
                const int j = at + __popc(m & ((1u << tid) - 1u));
                from[j] = s;
                to[j] = d;
            }
            at += __popc(m);
            __syncwarp();
        }
        if (tid == 0) count = at;
    }
    __syncthreads();
    const int moves = count;
    if (moves == 0) return;
    // Items in turn, the next one's sources requested before the last one's are written: while an item's writes go
    // out, the next one's reads come in.
    int64_t next = blockIdx.x, base = 0;                // the next item, and the first one of its buffer
    int buffer = 0;
    struct Item {
        uint8_t* data;
        int64_t bytes, at;
        int len;                                        // 16-byte pieces of a page; 0: no item
    };
    auto take = [&]() {
        Item it{nullptr, 0, 0, 0};
        while (buffer < b.n) {
            const int64_t items = (b.bytes[buffer] + range - 1) / range;
            if (next - base < items) {
                it.data = b.data[buffer];
                it.bytes = b.bytes[buffer];
                it.at = (next - base) * range;
                it.len = (int)min((int64_t)range, it.bytes - it.at) >> 4;
                next += gridDim.x;
                break;
            }
            base += items;
            ++buffer;
        }
        return it;
    };
    auto request = [&](const Item& it, uint8_t* room) {
        const int pieces = moves * it.len;
        for (int p = tid; p < pieces; p += kCopyThreads) {
            const int i = p / it.len, c = p - i * it.len;
            cp_async16(smem_addr(room) + p * 16, it.data + from[i] * it.bytes + it.at + c * 16);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    Item cur = take();
    int odd = 0;
    request(cur, stage);
    while (cur.len > 0) {
        const Item ahead = take();
        request(ahead, stage + (size_t)(odd ^ 1) * n * range);
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        __syncthreads();
        const uint8_t* room = stage + (size_t)odd * n * range;
        const int pieces = moves * cur.len;
        for (int p = tid; p < pieces; p += kCopyThreads) {
            const int i = p / cur.len, c = p - i * cur.len;
            __stcs(reinterpret_cast<uint4*>(cur.data + to[i] * cur.bytes + cur.at + c * 16),
                   *reinterpret_cast<const uint4*>(room + (size_t)p * 16));
        }
        __syncthreads();
        cur = ahead;
        odd ^= 1;
    }
}

// ---- lists of moves ---------------------------------------------------------------------------------
// The workspace holds the number of moves and the moves (from, to); from = -1 writes zeros.
struct MoveList {
    int32_t* count;
    int32_t* from;
    int32_t* to;
};

MoveList move_list(void* workspace, int32_t n_slots) {
    int32_t* w = static_cast<int32_t*>(workspace);
    return {w, w + 4, w + 4 + n_slots};
}

constexpr int kPlanThreads = 1024;

// exclusive sum over the CTA's threads of `x` (0 or 1); the total in *total
GDN_DEVICE int block_rank(bool x, int* sums, int* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const unsigned m = __ballot_sync(0xffffffffu, x);
    if (lane == 0) sums[warp] = __popc(m);
    __syncthreads();
    int before = 0, all = 0;
    for (int w = 0; w < kPlanThreads / 32; ++w) {
        const int c = sums[w];
        before += w < warp ? c : 0;
        all += c;
    }
    __syncthreads();
    *total = all;
    return before + __popc(m & ((1u << lane) - 1u));
}

// fork: the valid entries, in order, take the lowest free slots, in order
__global__ void __launch_bounds__(kPlanThreads)
state_fork_plan_kernel(int32_t n_slots, int32_t* live, const int32_t* src, int32_t* dst, int32_t n, MoveList list) {
    __shared__ int sums[kPlanThreads / 32];
    grid_next();
    const int tid = threadIdx.x;
    // entries: -1 (a page of zeros) or a live slot
    int wanted = 0;
    for (int i0 = 0; i0 < n; i0 += kPlanThreads) {
        const int i = i0 + tid;
        const int32_t s = i < n ? src[i] : -2;
        const bool ok = s == -1 || (s >= 0 && s < n_slots && live[s] != 0);
        int all;
        const int r = block_rank(ok, sums, &all);
        if (i < n) dst[i] = -1;
        if (ok && wanted + r < n_slots) {
            list.from[wanted + r] = s;
            list.to[wanted + r] = i;               // the entry, for now
        }
        wanted += all;
    }
    if (wanted > n_slots) wanted = n_slots;
    __syncthreads();
    int got = 0;
    for (int s0 = 0; s0 < n_slots && got < wanted; s0 += kPlanThreads) {
        const int s = s0 + tid;
        const bool free_slot = s < n_slots && live[s] == 0;
        int all;
        const int r = got + block_rank(free_slot, sums, &all);
        if (free_slot && r < wanted) {
            dst[list.to[r]] = s;
            list.to[r] = s;
            live[s] = 1;
        }
        got += all;
    }
    if (tid == 0) *list.count = min(got, wanted);
}

// compact: the live slots from n_live on move into the free ones before it, both in order
__global__ void __launch_bounds__(kPlanThreads)
state_compact_plan_kernel(int32_t n_slots, int32_t* live, int32_t* moved, MoveList list) {
    __shared__ int sums[kPlanThreads / 32];
    grid_next();
    const int tid = threadIdx.x;
    int n_live = 0;
    for (int s0 = 0; s0 < n_slots; s0 += kPlanThreads) {
        int all;
        block_rank(s0 + tid < n_slots && live[s0 + tid] != 0, sums, &all);
        n_live += all;
    }
    int gaps = 0, late = 0;
    for (int s0 = 0; s0 < n_slots; s0 += kPlanThreads) {
        const int s = s0 + tid;
        const bool is_live = s < n_slots && live[s] != 0;
        const bool gap = s < n_live && !is_live, is_late = s >= n_live && is_live;
        int all;
        const int g = block_rank(gap, sums, &all);
        if (gap) list.to[gaps + g] = s;
        gaps += all;
        const int r = block_rank(is_late, sums, &all);
        if (is_late) list.from[late + r] = s;
        late += all;
        if (s < n_slots) {
            moved[s] = is_live ? s : -1;
            live[s] = s < n_live ? 1 : 0;
        }
    }
    __syncthreads();
    for (int i = tid; i < late; i += kPlanThreads) moved[list.from[i]] = list.to[i];
    if (tid == 0) *list.count = late;              // = gaps
}

// The moves of a list whose sources and destinations are disjoint: an item is
// 16 KB of one page, neighbouring items the same bytes of the next moves (a
// source that several entries share is then read from memory once; taking the
// pages' bytes at different places at a time was up to 40% slower).  Moving 21
// pages of 77 MB down and starting 21: 5.9 TB/s; 32 pages from three: 5.4 TB/s
// (items of 32 KB in 256 threads: 5.6 and 4.9).
constexpr int kMoveThreads = 128;
constexpr int kMoveLoads = 8;
constexpr int kMoveBytes = kMoveThreads * kMoveLoads * 16;
constexpr int kMoveCtas = 16;                  // per SM

__global__ void __launch_bounds__(kMoveThreads) state_move_kernel(StateBuffers b, MoveList list) {
    grid_wait();
    const int64_t moves = *list.count;
    int64_t item = blockIdx.x;
    for (int k = 0; k < b.n; ++k) {
        const int64_t items = (b.bytes[k] + kMoveBytes - 1) / kMoveBytes * moves;
        for (; item < items; item += gridDim.x) {
            const int64_t range = item / moves;
            const int m = (int)(item - range * moves);
            const int32_t from = list.from[m];
            const int64_t at = range * kMoveBytes + threadIdx.x * 16;
            const uint8_t* s = b.data[k] + (int64_t)from * b.bytes[k] + at;
            uint8_t* d = b.data[k] + (int64_t)list.to[m] * b.bytes[k] + at;
            uint4 x[kMoveLoads];
#pragma unroll
            for (int j = 0; j < kMoveLoads; ++j) {
                x[j] = make_uint4(0u, 0u, 0u, 0u);
                if (from >= 0 && at + j * (kMoveThreads * 16) < b.bytes[k])
                    x[j] = *reinterpret_cast<const uint4*>(s + j * (kMoveThreads * 16));
            }
#pragma unroll
            for (int j = 0; j < kMoveLoads; ++j)
                if (at + j * (kMoveThreads * 16) < b.bytes[k])
                    __stcs(reinterpret_cast<uint4*>(d + j * (kMoveThreads * 16)), x[j]);
        }
        item -= items;
    }
}

__global__ void state_free_kernel(int32_t* live, int32_t n_slots, const int32_t* slots, int32_t n) {
    const int i = blockIdx.x * blockDim.x + threadIdx.x;
    if (i < n && slots[i] >= 0 && slots[i] < n_slots) live[slots[i]] = 0;
}

cudaError_t launch_moves(const StateBuffers& b, const MoveList& list, int64_t most, Chain& chain) {
    int64_t items = 0;
    for (int k = 0; k < b.n; ++k) items += (b.bytes[k] + kMoveBytes - 1) / kMoveBytes * most;
    if (items == 0) return cudaSuccess;
    const int64_t grid = items < 148 * kMoveCtas ? items : 148 * kMoveCtas;
    return chain.launch(true, state_move_kernel, (unsigned)grid, kMoveThreads, 0, b, list);
}

}  // namespace

size_t state_workspace_bytes(int32_t n_slots) { return (16 + (size_t)n_slots * 8 + 255) & ~(size_t)255; }

cudaError_t launch_state_copy(const StateBuffers& b, const int32_t* src, const int32_t* dst, int32_t n,
                              cudaStream_t s) {
    // The range of a page per item: what fits the room, in whole lines, or less where that would leave SMs without an
    // item (down to 1 KB); with more than 832 entries half a line.
    constexpr int kSms = 148;
    int64_t page = 0, items = 0;
    for (int k = 0; k < b.n; ++k) page += b.bytes[k];
    int range = kCopyStage / n / kCopyStep * kCopyStep;
    if (range > kCopyMostRange) range = kCopyMostRange;
    const int64_t share = page / kSms / kCopyStep * kCopyStep;
    if (range > share) range = share > 1024 ? (int)share : range < 1024 ? range : 1024;
    if (range == 0) range = kCopyMinRange;
    for (int k = 0; k < b.n; ++k) items += (b.bytes[k] + range - 1) / range;
    if (items == 0) return cudaSuccess;
    const size_t smem = 2 * (size_t)n * range + (size_t)n * 8;
    // (one limit for every call: two at once must not lower it for each other)
    cudaError_t e = cudaFuncSetAttribute(state_copy_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kCopyMostSmem);
    if (e != cudaSuccess) return e;
    const int64_t grid = items < kSms ? items : kSms;
    state_copy_kernel<<<(unsigned)grid, kCopyThreads, smem, s>>>(b, src, dst, n, range);
    return cudaGetLastError();
}

cudaError_t launch_state_fork(const StateBuffers& b, int32_t* live, const int32_t* src, int32_t* dst, int32_t n,
                              void* workspace, cudaStream_t s) {
    const MoveList list = move_list(workspace, b.n_slots);
    Chain chain{s};
    const cudaError_t e = chain.launch(false, state_fork_plan_kernel, 1, kPlanThreads, 0, b.n_slots, live, src, dst, n, list);
    return e == cudaSuccess ? launch_moves(b, list, n < b.n_slots ? n : b.n_slots, chain) : e;
}

cudaError_t launch_state_compact(const StateBuffers& b, int32_t* live, int32_t* moved, void* workspace,
                                 cudaStream_t s) {
    const MoveList list = move_list(workspace, b.n_slots);
    Chain chain{s};
    const cudaError_t e = chain.launch(false, state_compact_plan_kernel, 1, kPlanThreads, 0, b.n_slots, live, moved, list);
    return e == cudaSuccess ? launch_moves(b, list, b.n_slots / 2, chain) : e;
}

cudaError_t launch_state_free(int32_t* live, int32_t n_slots, const int32_t* slots, int32_t n, cudaStream_t s) {
    if (n == 0) return cudaSuccess;
    state_free_kernel<<<(n + 127) / 128, 128, 0, s>>>(live, n_slots, slots, n);
    return cudaGetLastError();
}

}  // namespace gdn
