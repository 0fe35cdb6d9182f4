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
#include "host.h"
#include "lola_internal.h"

namespace lola {

struct KeySeg {            // one segment of keys; strides in elements
    const void* k;
    const void* v;
    long long kb, ks, kh, vb, vs, vh;    // batch (0: shared), token, head
    int n;                               // keys (per sequence)
};

enum class AttnBy { none, rows, tiles };

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
    // How the work is cut (plan_attn).  A part is what one CTA makes of a row: its sum over a
    // range of keys.  With one part the CTA writes y; else it leaves the normalised sum and
    // its log2-sum-exp in the workspace and attn_join_kernel puts the parts together.
    int walk;              // 1: a sequence's rows read the shared keys too, before their own;
                           // 0: the shared keys are read by all sequences' rows as one group
    AttnBy by_shared, by_own;          // the kernels of the group over all sequences and of each sequence
    int parts_shared, parts_own;       // parts of a row from each (0: that kernel has nothing to do)
    int chunk_shared, chunk_own;       // keys per part
    float* part_o;         // [parts][B T Hq][d]
    float* part_l;         // [parts][B T Hq]
    // attn_rows_kernel with each kv head's rounds dealt evenly to this many CTAs (0: a CTA per group): what is
    // left of groups that a cut goes through, and the rounds before each sequence
    int even, slot_rows, beside;       // beside: on SMs that the shared keys' tiles leave free, at the same time
    float* slot_o;         // [even][Hkv][2][slot_rows][d]
    float* slot_l;         // [even][Hkv][2][slot_rows]
    int* goff;             // [B + 1]
};
constexpr int kRwRound = 64;           // keys of a round

// Chooses how the keys are cut (every field after scale_log2 but the pointers) and returns the
// bytes of workspace that needs.
size_t plan_attn(AttnArgs& a, int num_sms);
void place_attn(AttnArgs& a, void* workspace);       // sets the pointers into it
cudaError_t launch_attn(const AttnArgs& a, int num_sms, int* launches, cudaStream_t s);
// bf16, up to kRowsMax rows per group (attn_rows.cu); the parts of both kinds that are its own
constexpr int kRowsMax = 16;
cudaError_t launch_attn_rows(const AttnArgs& a, cudaStream_t s);   // (a.beside: behind launch_attn_tc)
// bf16, any number of rows, 128 keys at a time (attn_tc.cu); the parts of both kinds that are its own
cudaError_t launch_attn_tc(const AttnArgs& a, int num_sms, cudaStream_t s);
// f32 (attn_f32.cu): up to kF32RowsMax rows of a sequence; any number of rows, packed: the shared keys' group
constexpr int kF32RowsMax = 16;
cudaError_t launch_attn_f32_rows(const AttnArgs& a, cudaStream_t s);
cudaError_t launch_attn_f32_tiles(const AttnArgs& a, int packed, cudaStream_t s);
cudaError_t attn_error_word(int* word, cudaStream_t s);

// Programmatic dependent launch inside one call: a kernel launched `behind` another may begin before that one
// has ended (its begin and first loads hide behind the other's end), and waits with attn_wait_before where it
// needs what that one wrote.  The first kernel of a call is launched in plain stream order, so nothing of a call
// begins before earlier work on the stream has ended.  attn_let_next_begin: the next kernel may be scheduled.
__device__ __forceinline__ void attn_wait_before() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void attn_let_next_begin() { asm volatile("griddepcontrol.launch_dependents;"); }
template <typename Args>
cudaError_t attn_launch(void (*kernel)(const Args), unsigned grid, unsigned threads, size_t smem, bool behind, cudaStream_t s,
                        const Args& args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = behind ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, args);
}

// Where row r of a group is: its token over the batch, its offset in q (elements), its index in y.
struct RowAt {
    int n, t;
    long long q;
    size_t o;
};
__device__ __forceinline__ RowAt row_at(const AttnArgs& a, int n0, int g, int r) {
    RowAt x;
    x.n = n0 + r / a.Gq;
    const int h = g * a.Gq + r % a.Gq, b = x.n / a.T;
    x.t = x.n - b * a.T;
    x.q = b * a.qb + x.t * a.qs + h * a.qh;
    x.o = (size_t)x.n * a.Hq + h;
    return x;
}
__device__ __forceinline__ int own_length(const AttnArgs& a, int b) {
    return a.own_len ? min(max(a.own_len[b], 0), a.own.n) : a.own.n;
}
// own keys that query t reads, of a sequence that has len
__device__ __forceinline__ int own_visible(const AttnArgs& a, int len, int t) {
    return a.causal ? min(len, max(0, len - a.T + t + 1)) : len;
}

}  // namespace lola
