// Exact attention beside the hybrid layer: arguments shared by its kernels and
// its C entry points.
//
// Rows and groups.  All query heads of one kv head read the same keys, so the
// unit of work is a row (token, head of the kv group).  With n = the token's
// index over the batch (n = b T + t), row r = n Gq + (head in the group).
// The keys shared by the batch are read by all B T Gq rows of a kv head as one
// group; a sequence's own keys by its T Gq rows.  Both segments of a row enter
// one softmax: they are either walked one after the other by the same CTA, or
// reduced apart and joined by their log-sum-exp.
#pragma once
#include "lola_internal.h"

namespace lola {

struct KeySeg {            // one segment of keys; strides in elements
    const void* k;
    const void* v;
    long long kb, ks, kh, vb, vs, vh;    // batch (0: shared), token, head
    int n;                               // keys (per sequence)
};

struct AttnArgs {
    const void* q;
    long long qb, qs, qh;
    void* y;               // [B][T][Hq][d] in dtype
    float* lse;            // [B][T][Hq] or null: natural log of the row's sum of exp(scale q.k)
    KeySeg shared;         // n = 0: none
    KeySeg own;            // n = 0: none
    const int* own_len;    // [B] device, or null: own.n keys of every sequence
    int causal;            // query t reads own keys s <= len - T + t (else s < len)
    int B, T, Hq, Hkv, Gq, d, dtype;
    float scale_log2;      // scale * log2(e)
};

cudaError_t launch_attn(const AttnArgs& a, cudaStream_t s);

}  // namespace lola
