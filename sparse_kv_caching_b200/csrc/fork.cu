// Copies of whole sequences between (or inside) layer states: sequence b of the
// destination takes every memory of sequence parents[b] of the source
// (samples of one prompt, the surviving beams of a search step, the sequences
// that are not finished).  A sequence's part of one memory is a contiguous
// run of Hkv streams, so a memory is a matrix of sequences x columns and the
// fork is a gather of its rows: x'[b][c] = x[parents[b]][c].
//
// Bound: HBM.  It reads each distinct parent once and writes each sequence
// once; nothing is computed.  A thread owns one column (16 bytes; 4 where a
// sequence's run is not a multiple of 16) and moves it for many sequences.
//
// * Between two states: loads and stores of kBatch sequences at a time; a run of
//   sequences with one parent reads it once (samples of a prompt are such a
//   run), other repeats come from L2.
// * Inside one state the gather overwrites its own sources, in any pattern
//   (a swap, a cycle, two children).  The thread that owns a column first
//   reads it for every sequence that moves into its own shared-memory
//   slots, then writes them: no barrier, no second buffer and no order of
//   moves is needed, and sequences that stay are not touched.
#include "lola_internal.h"

namespace lola {

constexpr int kForkBatch = 8;          // sequences in flight per thread

// The index arithmetic of both kernels: tile -> segment and first column.
__device__ __forceinline__ const ForkSeg& fork_seg(const ForkArgs& a, long long tile, long long& col0) {
    int i = 0;
    while (i + 1 < a.nseg && tile >= a.seg[i + 1].tile0) ++i;
    col0 = (tile - a.seg[i].tile0) * a.tile_cols;
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
__global__ void __launch_bounds__(256) fork_kernel(const __grid_constant__ ForkArgs a) {
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
__device__ __forceinline__ void fork_stage_col(const ForkSeg& sg, const int* to, const int* from, int m, V* slot,
                                               long long col) {
    char* base = sg.dst + col * sizeof(V);
    const int nt = blockDim.x;
    for (int i0 = 0; i0 < m; i0 += kForkBatch) {
        V x[kForkBatch];
#pragma unroll
        for (int u = 0; u < kForkBatch; ++u)
            if (i0 + u < m) x[u] = *reinterpret_cast<const V*>(base + from[i0 + u] * sg.seq_bytes);
#pragma unroll
        for (int u = 0; u < kForkBatch; ++u)
            if (i0 + u < m) slot[(i0 + u) * nt] = x[u];
    }
    for (int i = 0; i < m; ++i) *reinterpret_cast<V*>(base + to[i] * sg.seq_bytes) = slot[i * nt];
}

// Inside one state (src == dst).  Shared memory: [n] to, [n] from, then the slots.
__global__ void fork_in_place_kernel(const __grid_constant__ ForkArgs a) {
    extern __shared__ __align__(16) unsigned char fork_smem[];
    __shared__ int moved;
    const int nt = blockDim.x, tid = threadIdx.x, n4 = (a.n + 3) & ~3;
    int* to = reinterpret_cast<int*>(fork_smem);
    int* from = to + n4;
    unsigned char* slots = fork_smem + 2 * n4 * sizeof(int);
    if (tid == 0) moved = 0;
    __syncthreads();
    bool bad = false;
    for (int b = tid; b < a.n; b += nt) {
        const int p = a.parents[b];
        const bool out = p < 0 || p >= a.src_B;
        bad |= out;
        if (!out && p != b) {
            const int i = atomicAdd(&moved, 1);        // any order: the moves are independent once staged
            to[i] = b;
            from[i] = p;
        }
    }
    fork_flags(a, bad);
    __syncthreads();
    const int m = moved;
    for (long long tile = blockIdx.x; tile < a.tiles; tile += gridDim.x) {
        long long col0;
        const ForkSeg& sg = fork_seg(a, tile, col0);
        const long long col = col0 + tid;
        if (col >= sg.cols) continue;
        if (sg.wide) fork_stage_col(sg, to, from, m, reinterpret_cast<uint4*>(slots) + tid, col);
        else fork_stage_col(sg, to, from, m, reinterpret_cast<uint32_t*>(slots) + tid, col);
    }
}

// The widest in-place launch whose slots fit: 16-byte columns while 32 threads'
// slots do, else 4-byte columns (n up to kForkInPlaceMax).
static void in_place_shape(int n, int* threads, int* col_bytes, size_t* smem) {
    const size_t budget = 200 * 1024, idx = 2 * (size_t)((n + 3) & ~3) * sizeof(int);
    *col_bytes = 16;
    *threads = 128;
    // up to a third of an SM's shared memory per CTA, so that three share it
    while (*threads > 32 && idx + (size_t)n * *threads * 16 > 68 * 1024) *threads >>= 1;
    if (idx + (size_t)n * *threads * 16 > budget) *col_bytes = 4;
    *smem = idx + (size_t)n * *threads * *col_bytes;
}

cudaError_t launch_fork(ForkArgs a, int num_sms, cudaStream_t s) {
    const bool in_place = a.seg[0].src == a.seg[0].dst;
    int threads = 256, col_bytes = 16;
    size_t smem = 0;
    if (in_place) in_place_shape(a.n, &threads, &col_bytes, &smem);
    a.tile_cols = threads;
    a.tiles = 0;
    for (int i = 0; i < a.nseg; ++i) {
        ForkSeg& sg = a.seg[i];
        sg.wide = col_bytes == 16 && sg.seq_bytes % 16 == 0;
        sg.cols = sg.seq_bytes / (sg.wide ? 16 : 4);
        sg.tile0 = a.tiles;
        a.tiles += (sg.cols + threads - 1) / threads;
    }
    const long long most = (long long)num_sms * 32;
    const unsigned gx = (unsigned)(a.tiles < most ? a.tiles : most);
    if (!in_place) {
        fork_kernel<<<dim3(gx, (a.n + kForkGroup - 1) / kForkGroup), threads, 0, s>>>(a);
        return cudaGetLastError();
    }
    cudaError_t e = cudaFuncSetAttribute(fork_in_place_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    fork_in_place_kernel<<<gx, threads, smem, s>>>(a);
    return cudaGetLastError();
}

}  // namespace lola
