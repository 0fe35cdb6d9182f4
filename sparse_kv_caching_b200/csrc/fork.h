// Copies of whole sequences (fork.cu): what the entry point hands to the launcher.
#pragma once
#include <cuda_runtime.h>

namespace lola {

// One memory of a fork: rows of seq_bytes, one per sequence, gathered by the parents.
struct ForkSeg {
    const char* src;
    char* dst;
    long long seq_bytes;
    long long cols, tile0; // columns per sequence and the memory's first tile (set by the launcher)
    int wide;              // columns of 16 bytes (else 4)
};
constexpr int kForkSegs = 13;          // memories a fork may copy
constexpr int kForkGroup = 64;         // destination sequences per CTA (between two states)
constexpr int kForkInPlaceMax = 1500;  // sequences of an in-place fork (shared-memory slots, 32 threads x 4 bytes)

struct ForkArgs {
    ForkSeg seg[kForkSegs];
    int nseg;
    const int* parents;    // [n] device
    int n, src_B;
    int* src_err;
    int* dst_err;          // bit 1: a parent outside [0, src_B)
    long long tiles;       // set by the launcher, as
    int wide;              // in place: 16-byte slots (else 4)
};

cudaError_t launch_fork(ForkArgs a, int num_sms, cudaStream_t s);

}  // namespace lola
