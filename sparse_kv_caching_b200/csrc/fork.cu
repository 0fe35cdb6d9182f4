// Copies of whole sequences between (or inside) layer states: sequence b of the
// destination takes every memory of sequence parents[b] of the source
// (samples of one prompt, the surviving beams of a search step, the sequences
// that are not finished).  A sequence's part of one memory is a contiguous
// run of Hkv streams, so a memory is a matrix of sequences x columns and the
// fork is a gather of its rows: x'[b][c] = x[parents[b]][c].
//
// Bound: HBM.  It reads each distinct parent once and writes each sequence
// once; nothing is computed.  A thread owns one column (16 bytes; 4 where a
// sequence's run is not a multiple of 16) and moves it for many sequences, eight
// loads in flight.  B200, the 8B-shaped decode layer (3.2 MB a sequence): one prompt
// to 64 sequences 37.5 us, 205 MB, 5.5 TB/s (a plain fill of as much takes 31);
// 44 of 64 beams from 20 survivors in place 57.5 us for 270 MB (decode's residuals
// included), 4.7 TB/s.  16 loads in flight spill (50 and 96 us); 128-thread CTAs 39
// and 63; moves sorted by parent so that equal ones share a load 89 in place.
//
// * Between two states: loads and stores of kBatch sequences at a time; a run of
//   sequences with one parent reads it once (samples of a prompt are such a
//   run), other repeats come from L2.
// * Inside one state the gather may overwrite its own sources, in any pattern (a
//   swap, a cycle, two children).  Sequences that move and are a parent of
//   another are the hazards: the thread that owns a column first reads it for every
//   hazard into its own shared-memory slots, then makes the moves, reading
//   hazards from the slots and all other parents (which stay, or are no
//   destination) where they lie.  No barrier, no second buffer and no order of
//   moves is needed, and sequences that stay are not touched.  A search step that
//   replaces dead beams by survivors has no hazards and runs with every thread; with
//   many hazards a CTA's first threads share all of its slots.
#include <limits.h>

#include "fork.h"
#include "host.h"

namespace lola {

constexpr int kForkBatch = 8;          // sequences in flight per thread
constexpr int kForkThreads = 256;      // columns of a tile

// The index arithmetic of both kernels: tile -> segment and first column.
__device__ __forceinline__ const ForkSeg& fork_seg(const ForkArgs& a, long long tile, long long& col0) {
    int i = 0;
    while (i + 1 < a.nseg && tile >= a.seg[i + 1].tile0) ++i;
    col0 = (tile - a.seg[i].tile0) * kForkThreads;
    return a.seg[i];
}

__device__ __forceinline__ void fork_flags(const ForkArgs& a, bool bad) {
    if (bad) atomicOr(a.dst_err, 2);
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0 && a.src_err != a.dst_err) {
        const int e = *a.src_err;      // a source that is not valid makes copies that are not valid
        if (e) atomicOr(a.dst_err, e);
    }
}

template <typename V>
__device__ __forceinline__ void fork_copy_col(const ForkArgs& a, const ForkSeg& sg, const int* par, int b0, int nb,
                                              long long col) {
    const char* src = sg.src + col * sizeof(V);
    char* dst = sg.dst + b0 * sg.seq_bytes + col * sizeof(V);
    for (int i0 = 0; i0 < nb; i0 += kForkBatch) {
        V x[kForkBatch];
#pragma unroll
        for (int u = 0; u < kForkBatch; ++u) {
            if (i0 + u >= nb) break;
            const int p = par[i0 + u];
            if (u > 0 && p == par[i0 + u - 1]) x[u] = x[u - 1];
            else if (p >= 0) x[u] = *reinterpret_cast<const V*>(src + p * sg.seq_bytes);
        }
#pragma unroll
        for (int u = 0; u < kForkBatch; ++u)
            if (i0 + u < nb && par[i0 + u] >= 0) *reinterpret_cast<V*>(dst + (i0 + u) * sg.seq_bytes) = x[u];
    }
}

// Between two states: blockIdx.y picks kForkGroup destination sequences.
__global__ void __launch_bounds__(kForkThreads, 3) fork_kernel(const __grid_constant__ ForkArgs a) {
    __shared__ int par[kForkGroup];
    const int b0 = blockIdx.y * kForkGroup, nb = min(kForkGroup, a.n - b0);
    bool bad = false;
    if (threadIdx.x < nb) {
        int p = a.parents[b0 + threadIdx.x];
        bad = p < 0 || p >= a.src_B;
        par[threadIdx.x] = bad ? -1 : p;
    }
    fork_flags(a, bad);
    __syncthreads();
    for (long long tile = blockIdx.x; tile < a.tiles; tile += gridDim.x) {
        long long col0;
        const ForkSeg& sg = fork_seg(a, tile, col0);
        const long long col = col0 + threadIdx.x;
        if (col >= sg.cols) continue;
        if (sg.wide) fork_copy_col<uint4>(a, sg, par, b0, nb, col);
        else fork_copy_col<uint32_t>(a, sg, par, b0, nb, col);
    }
}

template <typename V>
__device__ __forceinline__ void fork_move_col(const ForkSeg& sg, const int* to, const int* from, int m, const int* hazard,
                                              int h, V* slot, int nt, long long col) {
    char* base = sg.dst + col * sizeof(V);
    for (int i0 = 0; i0 < h; i0 += kForkBatch) {
        V x[kForkBatch];
#pragma unroll
        for (int u = 0; u < kForkBatch; ++u)
            if (i0 + u < h) x[u] = *reinterpret_cast<const V*>(base + hazard[i0 + u] * sg.seq_bytes);
#pragma unroll
        for (int u = 0; u < kForkBatch; ++u)
            if (i0 + u < h) slot[(i0 + u) * nt] = x[u];
    }
    for (int i0 = 0; i0 < m; i0 += kForkBatch) {
        V x[kForkBatch];
#pragma unroll
        for (int u = 0; u < kForkBatch; ++u)
            if (i0 + u < m) {
                const int p = from[i0 + u];       // a sequence, or -1 - slot
                x[u] = p >= 0 ? *reinterpret_cast<const V*>(base + p * sg.seq_bytes) : slot[(-1 - p) * nt];
            }
#pragma unroll
        for (int u = 0; u < kForkBatch; ++u)
            if (i0 + u < m) *reinterpret_cast<V*>(base + to[i0 + u] * sg.seq_bytes) = x[u];
    }
}

// Inside one state (src == dst).  Shared memory: [n] parent, [n] to, [n] from, [n] hazard, then the slots.
__global__ void __launch_bounds__(kForkThreads, 2) fork_in_place_kernel(const __grid_constant__ ForkArgs a, int slot_bytes) {
    extern __shared__ __align__(16) unsigned char fork_smem[];
    __shared__ int moved, hazards;
    const int tid = threadIdx.x, n4 = (a.n + 3) & ~3;
    int* par = reinterpret_cast<int*>(fork_smem);
    int *to = par + n4, *from = to + n4, *hazard = from + n4;
    unsigned char* slots = fork_smem + 4 * n4 * sizeof(int);
    if (tid == 0) moved = hazards = 0;
    bool bad = false;
    for (int b = tid; b < a.n; b += kForkThreads) {
        const int p = a.parents[b];
        const bool out = p < 0 || p >= a.src_B;
        bad |= out;
        par[b] = out ? b : p;
        to[b] = 0;                                // (until the lists are made: 1 where b is a parent of another)
    }
    fork_flags(a, bad);
    __syncthreads();
    for (int b = tid; b < a.n; b += kForkThreads)
        if (par[b] != b && par[b] < a.n) to[par[b]] = 1;
    __syncthreads();
    for (int b = tid; b < a.n; b += kForkThreads) {
        from[b] = 0;
        if (to[b] && par[b] != b) {
            const int i = atomicAdd(&hazards, 1); // any order: slots do not depend on each other
            hazard[i] = b;
            from[b] = -1 - i;                     // (for the moment: by sequence)
        }
    }
    __syncthreads();
    const int h = hazards;
    // this thread's moves, from the table by sequence to the lists
    constexpr int kMost = (kForkInPlaceMax + kForkThreads - 1) / kForkThreads;
    int src[kMost];
#pragma unroll
    for (int u = 0; u < kMost; ++u) {
        const int b = tid + u * kForkThreads;
        src[u] = b < a.n && par[b] != b ? (par[b] < a.n && from[par[b]] < 0 ? from[par[b]] : par[b]) : INT_MIN;
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kMost; ++u)
        if (src[u] != INT_MIN) {
            const int i = atomicAdd(&moved, 1);
            to[i] = tid + u * kForkThreads;
            from[i] = src[u];
        }
    __syncthreads();
    const int m = moved, width = a.wide ? 16 : 4;
    int nt = kForkThreads;                        // threads whose slots fit
    while (nt > 32 && nt * h * width > slot_bytes) nt >>= 1;
    if (m == 0 || tid >= nt) return;
    for (long long tile = blockIdx.x; tile < a.tiles; tile += gridDim.x) {
        long long col0;
        const ForkSeg& sg = fork_seg(a, tile, col0);
        const long long end = min(sg.cols, col0 + kForkThreads);
        for (long long col = col0 + tid; col < end; col += nt) {
            if (sg.wide) fork_move_col(sg, to, from, m, hazard, h, reinterpret_cast<uint4*>(slots) + tid, nt, col);
            else fork_move_col(sg, to, from, m, hazard, h, reinterpret_cast<uint32_t*>(slots) + tid, nt, col);
        }
    }
}

// Shared memory of an in-place fork of n sequences.  Every sequence may be a hazard: 32 threads' slots have
// to fit, 16 bytes wide up to 200 KB, else 4.  Up to 128 sequences that is the 64 KB with which three CTAs
// share an SM.
constexpr bool fork_wide(int n) { return n * 32 * 16 <= 200 * 1024; }
constexpr int fork_slot_bytes(int n) {
    const int b = n * 32 * (fork_wide(n) ? 16 : 4);
    return b > 64 * 1024 ? b : 64 * 1024;
}
constexpr int fork_smem_bytes(int n) { return 4 * ((n + 3) & ~3) * (int)sizeof(int) + fork_slot_bytes(n); }
constexpr int fork_smem_most() {
    int most = 0;
    for (int n = 1; n <= kForkInPlaceMax; ++n)
        if (fork_smem_bytes(n) > most) most = fork_smem_bytes(n);
    return most;
}
static_assert(fork_smem_most() + 64 <= 227 * 1024, "shared memory");

cudaError_t launch_fork(ForkArgs a, int num_sms, cudaStream_t s) {
    const bool in_place = a.seg[0].src == a.seg[0].dst;
    a.wide = fork_wide(a.n);
    a.tiles = 0;
    for (int i = 0; i < a.nseg; ++i) {
        ForkSeg& sg = a.seg[i];
        sg.wide = (a.wide || !in_place) && sg.seq_bytes % 16 == 0;
        sg.cols = sg.seq_bytes / (sg.wide ? 16 : 4);
        sg.tile0 = a.tiles;
        a.tiles += (sg.cols + kForkThreads - 1) / kForkThreads;
    }
    auto grid = [&](long long most) { return (unsigned)(a.tiles < most ? a.tiles : most); };
    if (!in_place) {
        const int groups = (a.n + kForkGroup - 1) / kForkGroup;
        fork_kernel<<<dim3(grid((3LL * num_sms + groups - 1) / groups), groups), kForkThreads, 0, s>>>(a);
        return cudaGetLastError();
    }
    static std::atomic<unsigned long long> done{0};
    cudaError_t e = allow_smem(fork_in_place_kernel, fork_smem_most(), &done);
    if (e != cudaSuccess) return e;
    fork_in_place_kernel<<<grid(3LL * num_sms), kForkThreads, fork_smem_bytes(a.n), s>>>(a, fork_slot_bytes(a.n));
    return cudaGetLastError();
}

}  // namespace lola
