// Exact attention for many rows per kv head (prompts, and the rows of a whole
// batch against its shared prefix) on the fifth-generation tensor cores, bf16.
//
// Mathematics: one pass over tiles of 128 keys with a running reference r of the
// softmax exponents.  S = Q K^T (tensor cores, f32); P = 2^(c S - r), c =
// scale log2(e), r = c m; l += row sums of P in f32; O += P V with P rounded to bf16 (its
// product's type; half a step, 2^-8 of each weight, averages out over the keys,
// while f16 weights would need V converted).  m is raised only when a row's
// maximum passes m + 8 / c, which keeps P below 2^8 and makes rescaling O rare.
//
// Bound: the tensor cores (4 d operations per row and key) and, as hard, the
// exponentials: a 128 x 128 tile costs 1056 cycles of products and 1024 of the
// special-function unit.  So one CTA per SM works on two 128-row tiles A and B in
// turn: while the warps of A turn S_A into P_A, the tensor cores run B's
// products.  Both tiles read the same key tiles, which halves the reads from L2.
//   warps 0-3 / 4-7  softmax and output of tile A / B; thread r owns row r
//   warp 8           loads K and V tiles with TMA into a ring (128-byte swizzle)
//   warp 9           issues the products
//   warps 10-11      gather the query rows of the next work item
// Tensor memory: S_A, S_B (128 columns each; P as bf16 pairs over its own S), O_A,
// O_B.  S_t(j + 1) overwrites P_t(j) right behind O_t += P_t(j) V(j) in the same
// in-order queue, so S(j + 1) ready also means that O_t may be rescaled.
// CTAs are persistent: the next item's queries and keys load during the last
// products and the output of this one.
// B200, 4 x 4096 queries against 4096 states, 32/8 heads: d 128 928 us, 1185 TFLOP/s in short runs
// (about 1000 under the power cap); d 64 790 us.  A pair of tiles takes 3450 cycles: per row
// tile 1650 from its scores to its weights beside the other's, 1500 from there to the next scores.
// Every wait is bounded; one that gives up raises a flag that ends all others of
// the CTA, and sets the device's error word.
#include <cuda.h>

#include "attn.h"
#include "device_common.cuh"
#include "umma.cuh"

namespace lola {

__device__ int g_attn_err;

constexpr int kTcRows = 128, kTcKeys = 128, kTcThreads = 384;

struct TcArgs {
    CUtensorMap map[4];             // shared keys and values, own keys and values
    AttnArgs a;
    // Two kinds of items: [0] rows of the whole batch against the shared keys, [1] rows of one sequence
    // against its own keys, the shared ones first where they are walked.
    int row_tiles[2];               // 256-row tile pairs per group
    int parts[2], chunk[2];         // parts of a row, key tiles per part
    int shared_items, items;        // the items of kind 0, of both
    int mh[4], mb[4];               // coordinate multipliers of the maps: 0 where one head (sequence) serves all
};

template <int DIM>
struct TcShape {
    static constexpr int QB = kTcRows * DIM * 2, ST = kTcKeys * DIM * 2, NST = 4;
    static constexpr int Q = 0, RING = 2 * QB, OUT = RING + NST * ST, MBAR = OUT + 8 * 2048;    // OUT: 32 rows x 64 bytes per warp
    static constexpr int NBAR = 2 * NST + 11;
    static constexpr int FLAG = MBAR + NBAR * 8, BYTES = FLAG + 16 + 1024;
    static_assert(BYTES <= 227 * 1024, "shared memory");
    // tensor memory, all 512 columns of it: S (and P) of row tile t at 128 t, O at 256 + 128 t
    static constexpr uint32_t TS = 0, TO = 256;
    // barriers
    static constexpr int FULL = 0, FREE = NST, QFULL = 2 * NST, QFREE = QFULL + 2, SFULL = QFREE + 2,
                         PFULL = SFULL + 2, OFULL = PFULL + 2, DONE = OFULL + 2;
};

__device__ __forceinline__ bool tc_wait(uint64_t* mbar, uint32_t parity, volatile int* abort) {
    if (umma::mbar_try_wait(mbar, parity)) return true;
    const long long t0 = clock64();               // (globaltimer takes too long to read for a wait this short)
    for (unsigned n = 1;; ++n) {
        if (umma::mbar_try_wait(mbar, parity)) return true;
        if ((n & 63) == 0) {
            if (*abort) return false;
            if (clock64() - t0 > 8000000000ll) { *abort = 1; return false; }
        }
    }
}
__device__ __forceinline__ float tc_ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t tc_pack(float lo, float hi) {
    __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&v);
}
__device__ __forceinline__ void tc_tma(void* dst, const CUtensorMap* map, uint64_t* mbar, int key, int h, int b) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2,%3,%4,%5,%6}], [%7];"
        :: "r"(umma::smem_addr(dst)), "l"(map), "r"(0), "r"(key), "r"(0), "r"(h), "r"(b), "r"(umma::smem_addr(mbar))
        : "memory");
}
__device__ __forceinline__ void tc_expect(uint64_t* mbar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" :: "r"(umma::smem_addr(mbar)), "r"(bytes) : "memory");
}

// The products' warp runs as a whole and elects the lane that issues, and every operand of a
// product is a constant or the same in all lanes (the ring's stage, the row tile and the tensor
// memory's columns are constants of the code that issues): the compiler then keeps them in
// warp-wide registers, where the instruction takes them.  With operands that it has to move there
// each product costs several more instructions, and beside the two busy softmax warps on the same
// scheduler 16 products of 128 x 128 x 16 took 2255 cycles instead of 1377 (1025 alone).
__device__ __forceinline__ bool tc_elect() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}\n" : "=r"(p));
    return p != 0;
}
template <int V> struct TcInt { static constexpr int v = V; };
__device__ __forceinline__ bool tc_wait_warp(uint64_t* mbar, uint32_t parity, volatile int* abort) {
    return __all_sync(0xffffffffu, tc_wait(mbar, parity, abort));
}

// One work item: up to 256 rows of a group against a range of key tiles.
struct TcItem {
    int g, b, n0, R, r0, part;      // kv head, sequence, first token, rows of the group, first row, part (in the workspace)
    int nt0, j0, j1, len;           // shared tiles of the walk, this part's tiles, own length
    bool two;                       // tile B holds rows
};
__device__ __forceinline__ TcItem tc_item(const TcArgs& p, int i) {
    const AttnArgs& a = p.a;
    TcItem x;
    const int own = i >= p.shared_items, row_tiles = p.row_tiles[own], parts = p.parts[own];
    if (own) i -= p.shared_items;
    const int rt = i % row_tiles;
    i /= row_tiles;
    const int k = i % parts;
    i /= parts;
    x.part = own ? a.parts_shared + k : k;
    x.g = i % a.Hkv;
    x.b = i / a.Hkv;                // (0 for the shared keys)
    x.n0 = x.b * a.T;
    x.R = (own ? 1 : a.B) * a.T * a.Gq;
    x.r0 = rt * 2 * kTcRows;
    const int last = min(x.R, x.r0 + 2 * kTcRows) - 1;
    x.two = last >= x.r0 + kTcRows;
    x.len = own ? own_length(a, x.b) : 0;
    x.nt0 = !own || a.walk ? (a.shared.n + kTcKeys - 1) / kTcKeys : 0;
    const int vis = own ? own_visible(a, x.len, last / a.Gq) : 0;
    const int nt = x.nt0 + (vis + kTcKeys - 1) / kTcKeys;
    x.j0 = min(nt, k * p.chunk[own]);
    x.j1 = min(nt, x.j0 + p.chunk[own]);
    return x;
}

template <int DIM>
__global__ void __launch_bounds__(kTcThreads, 1) attn_tc_kernel(const __grid_constant__ TcArgs p) {
    using Sh = TcShape<DIM>;
    using bf16 = __nv_bfloat16;
    constexpr int NST = Sh::NST;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (umma::smem_addr(smem_raw) & 1023u)) & 1023u);
    const AttnArgs& a = p.a;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    uint8_t* sQ = smem + Sh::Q;
    uint8_t* ring = smem + Sh::RING;
    uint64_t* mbar = reinterpret_cast<uint64_t*>(smem + Sh::MBAR);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Sh::FLAG);
    uint32_t* tptr = reinterpret_cast<uint32_t*>(smem + Sh::FLAG + 8);

    attn_let_next_begin();
    if (warp == 0) umma::tmem_alloc(tptr, 512);
    if (tid == 0) {
        for (int i = 0; i < Sh::NBAR; ++i) umma::mbar_init(&mbar[i], 1);
        for (int t = 0; t < 2; ++t) {
            umma::mbar_init(&mbar[Sh::QFULL + t], 64);
            umma::mbar_init(&mbar[Sh::PFULL + t], kTcRows);
        }
        *abort_flag = 0;
        umma::fence_mbar_init();
    }
    umma::fence_before_sync();
    __syncthreads();
    umma::fence_after_sync();
    const uint32_t tmem = *tptr;                // all of tensor memory: column 0
    if (tid == 0 && tmem != 0) *abort_flag = 1;
    // registers: 256 x 208 + 128 x 88 = the 384 x 168 of the launch
    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
        if (warp == 8) {
            // ---- K and V tiles: K(j), V(j), K(j + 1), ... into consecutive ring stages ----
            if (lane == 0) {
                unsigned n = 0;                       // tiles loaded so far
                bool ok = true;
                for (int i = blockIdx.x; i < p.items && ok; i += gridDim.x) {
                    const TcItem x = tc_item(p, i);
                    for (int jj = 2 * x.j0; jj < 2 * x.j1 && ok; ++jj, ++n) {
                        const int s = n % NST, j = jj >> 1;
                        if (n >= NST) ok = tc_wait(&mbar[Sh::FREE + s], (n / NST - 1) & 1, abort_flag);
                        if (!ok) break;
                        const bool sh = j < x.nt0;
                        const int which = (sh ? 0 : 2) + (jj & 1);
                        tc_expect(&mbar[Sh::FULL + s], Sh::ST);
                        tc_tma(ring + s * Sh::ST, &p.map[which], &mbar[Sh::FULL + s], (sh ? j : j - x.nt0) * kTcKeys,
                               x.g * p.mh[which], x.b * p.mb[which]);
                    }
                }
                if (!ok)                              // given up: the copies in flight still land in this CTA's memory
                    for (unsigned m = n > NST ? n - NST : 0; m < n; ++m)
                        (void)umma::mbar_wait(&mbar[Sh::FULL + m % NST], (m / NST) & 1, 1000000000ull);
            }
        } else if (warp == 9) {
            // ---- products ----
            constexpr uint32_t idS = umma::idesc(umma::kBF16, kTcRows, kTcKeys, false, false);
            constexpr uint32_t idO = umma::idesc(umma::kBF16, kTcRows, DIM, false, true);
            const uint64_t dQ = umma::sdesc_sw128(umma::smem_addr(sQ), 16, 1024);
            const uint64_t dK = umma::sdesc_sw128(umma::smem_addr(ring), 16, 1024);
            const uint64_t dV = umma::sdesc_sw128(umma::smem_addr(ring), kTcKeys * 128, 1024);
            // S of row tile T from the key tile in stage ST.  Q and K: a step of 16 dims is 32 bytes inside
            // a 128-byte half row, the next half 128 rows on.
            auto scores = [&](auto T, auto ST, bool last) {
                constexpr int t = decltype(T)::v, st = decltype(ST)::v;
                if (!tc_elect()) return;
                constexpr int q0 = t * (Sh::QB / 16), k0 = st * (Sh::ST / 16);
                // (a loop of few registers: unrolled, its descriptors would all be kept across the loop over the tiles)
#pragma unroll 1
                for (int h = 0; h < DIM / 64; ++h)
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks) {
                        const int step = h * kTcRows * 8 + ks * 2;
                        umma::mma_bf16(Sh::TS + 128 * t, dQ + (uint64_t)(q0 + step), dK + (uint64_t)(k0 + step), idS, h + ks > 0);
                    }
                umma::commit(&mbar[Sh::SFULL + t]);
                if (last) umma::commit(&mbar[Sh::QFREE + t]);
            };
            // O of row tile T (+)= P V, V in stage ST
            auto values = [&](auto T, auto ST, bool first, bool last) {
                constexpr int t = decltype(T)::v, st = decltype(ST)::v;
                if (!tc_elect()) return;
#pragma unroll 1
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int k4 = 0; k4 < kTcKeys / 32; ++k4) {
                        const int ks = h * (kTcKeys / 32) + k4;
                        umma::mma_f16_ts(Sh::TO + 128 * t, Sh::TS + 128 * t + 8 * ks, dV + (uint64_t)(st * (Sh::ST / 16) + ks * 128),
                                         idO, ks > 0 || !first);
                    }
                if (last) umma::commit(&mbar[Sh::OFULL + t]);
            };
            auto release = [&](auto ST) {
                if (tc_elect()) umma::commit(&mbar[Sh::FREE + decltype(ST)::v]);
            };
            auto wait = [&](int i, unsigned parity) { return tc_wait_warp(&mbar[i], parity & 1, abort_flag); };
            // Key tile number g of this CTA sits in stages 2 (g % 2) and 2 (g % 2) + 1.
            unsigned g = 0, np[2] = {0, 0}, nq[2] = {0, 0};
            bool ok = true;
            // the first scores of an item
            auto open = [&](auto PAR, int nr, int nt) {
                constexpr int par = decltype(PAR)::v;
                ok = wait(Sh::FULL + 2 * par, g >> 1);
                auto row_tile = [&](auto T) {
                    constexpr int t = decltype(T)::v;
                    if (t >= nr || !ok) return;
                    ok = wait(Sh::QFULL + t, nq[t]++);
                    if (!ok) return;
                    umma::fence_after_sync();
                    scores(TcInt<t>{}, TcInt<2 * par>{}, nt == 1);
                };
                row_tile(TcInt<0>{});
                row_tile(TcInt<1>{});
                if (ok) release(TcInt<2 * par>{});
            };
            // values of tile j (parity PAR) and scores of the next, row tile by row tile
            auto step = [&](auto PAR, int nr, int nt, int j) {
                constexpr int par = decltype(PAR)::v;
                const bool more = j + 1 < nt;
                ok = wait(Sh::FULL + 2 * par + 1, g >> 1);
                if (more && ok) ok = wait(Sh::FULL + 2 * (1 - par), (g + 1) >> 1);
                auto row_tile = [&](auto T) {
                    constexpr int t = decltype(T)::v;
                    if (t >= nr || !ok) return;
                    ok = wait(Sh::PFULL + t, np[t]++);
                    if (!ok) return;
                    umma::fence_after_sync();
                    values(TcInt<t>{}, TcInt<2 * par + 1>{}, j == 0, !more);
                    if (more) scores(TcInt<t>{}, TcInt<2 * (1 - par)>{}, j + 2 == nt);
                };
                row_tile(TcInt<0>{});
                row_tile(TcInt<1>{});
                if (!ok) return;
                release(TcInt<2 * par + 1>{});
                if (more) release(TcInt<2 * (1 - par)>{});
            };
            for (int i = blockIdx.x; i < p.items && ok; i += gridDim.x) {
                const TcItem x = tc_item(p, i);
                const int nt = x.j1 - x.j0, nr = x.two ? 2 : 1;
                if (nt == 0) continue;
                if (g & 1) open(TcInt<1>{}, nr, nt);
                else open(TcInt<0>{}, nr, nt);
                for (int j = 0; j < nt && ok; ++j, ++g) {
                    if (g & 1) step(TcInt<1>{}, nr, nt, j);
                    else step(TcInt<0>{}, nr, nt, j);
                }
            }
            if (tc_elect()) umma::commit(&mbar[Sh::DONE]);        // nothing may be in flight when tensor memory is given back
            if (!umma::mbar_wait(&mbar[Sh::DONE], 0, 4000000000ull)) *abort_flag = 1;
        } else {
            // ---- queries: 128-byte swizzled, block kb holds dims 64 kb .. 64 kb + 63 of every row ----
            constexpr int NC = DIM / 8;
            unsigned nq[2] = {0, 0};
            bool ok = true;
            for (int i = blockIdx.x; i < p.items && ok; i += gridDim.x) {
                const TcItem x = tc_item(p, i);
                if (i + gridDim.x < p.items) {
                    // the next item's rows into L2 meanwhile: its copies start when this item's last scores are
                    // made, and the products wait for them
                    const TcItem y = tc_item(p, i + gridDim.x);
                    for (int R = y.r0 + tid - 320; R < min(y.R, y.r0 + 2 * kTcRows); R += 64) {
                        const bf16* q = (const bf16*)a.q + row_at(a, y.n0, y.g, R).q;
#pragma unroll
                        for (int c = 0; c < DIM; c += 64) asm volatile("prefetch.global.L2 [%0];" :: "l"(q + c));
                    }
                }
                if (x.j0 == x.j1) continue;
                for (int t = 0; t < (x.two ? 2 : 1) && ok; ++t) {
                    if (nq[t]) ok = tc_wait(&mbar[Sh::QFREE + t], (nq[t] - 1) & 1, abort_flag);
                    ++nq[t];
                    if (!ok) break;
                    // each lane finds one row, then 32 / NC rows at a time are copied in 16-byte chunks
#pragma unroll 1
                    for (int r32 = 32 * (warp - 10); r32 < kTcRows; r32 += 64) {
                        const int R = x.r0 + t * kTcRows + r32 + lane;
                        const long long at = R < x.R ? row_at(a, x.n0, x.g, R).q : -1;
#pragma unroll
                        for (int k = 0; k < NC; ++k) {
                            const int rr = k * (32 / NC) + lane / NC, c = lane % NC, r = r32 + rr;
                            const long long from = __shfl_sync(0xffffffffu, at, rr);
                            umma::cp_async16_zfill(sQ + t * Sh::QB + (c >> 3) * (kTcRows * 128) + umma::sw128_off(r, c & 7),
                                                   (const bf16*)a.q + (from < 0 ? 0 : from) + 8 * c, from >= 0);
                        }
                    }
                    umma::cp_async_commit();
                }
                if (!ok) break;
                if (x.two) {
                    umma::cp_async_wait<1>();
                    umma::fence_async_smem();
                    umma::mbar_arrive(&mbar[Sh::QFULL]);
                }
                umma::cp_async_wait<0>();
                umma::fence_async_smem();
                umma::mbar_arrive(&mbar[Sh::QFULL + (x.two ? 1 : 0)]);
            }
            umma::cp_async_wait<0>();
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
        // ---- softmax and output of row tile t ----
        const int t = warp >> 2, r = tid & (kTcRows - 1);
        const uint32_t lane_off = (uint32_t)(32 * (warp & 3)) << 16;
        const uint32_t tS = tmem + lane_off + Sh::TS + 128 * t, tO = tmem + lane_off + Sh::TO + 128 * t;
        const float c2 = a.scale_log2;
        unsigned n = 0, ns = 0, no = 0;           // ring position; tiles and items of this row tile
        bool dead = false;
        for (int i = blockIdx.x; i < p.items && !dead; i += gridDim.x) {
            const TcItem x = tc_item(p, i);
            if (t == 1 && !x.two) { n += 2 * (x.j1 - x.j0); continue; }
            const int R = x.r0 + t * kTcRows + r;
            const bool row_ok = R < x.R;
            const int vis = row_ok ? own_visible(a, x.len, row_at(a, x.n0, x.g, R).t) : 0, vis0 = row_ok ? a.shared.n : 0;
            float m = -INFINITY, l = 0.f;
            for (int j = x.j0; j < x.j1; ++j, ++ns) {
                bool ok = tc_wait(&mbar[Sh::SFULL + t], ns & 1, abort_flag);
                if (!__all_sync(0xffffffffu, ok)) { dead = true; break; }
                umma::fence_after_sync();
                float s[kTcKeys];
#pragma unroll
                for (int c = 0; c < kTcKeys; c += 16) umma::tmem_ld16(tS + c, *reinterpret_cast<float(*)[16]>(s + c));
                umma::tmem_wait_ld();
                const bool sh = j < x.nt0;
                const int k0 = (sh ? j : j - x.nt0) * kTcKeys, lim = (sh ? vis0 : vis) - k0;
                if (!__all_sync(0xffffffffu, lim >= kTcKeys)) {
#pragma unroll
                    for (int u = 0; u < kTcKeys; ++u) s[u] = u < lim ? s[u] : -INFINITY;
                }
                float m4[4] = {s[0], s[1], s[2], s[3]};      // four chains: the latency of one would show
#pragma unroll
                for (int u = 4; u < kTcKeys; u += 8)
#pragma unroll
                    for (int v = 0; v < 4; ++v) m4[v] = fmaxf(m4[v], u + 4 < kTcKeys ? fmaxf(s[u + v], s[u + v + 4]) : s[u + v]);
                const float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
                float f = 1.f;
                bool raise = false;
                if (m == -INFINITY) m = mx;       // nothing read yet
                else if ((mx - m) * c2 > 8.f) {
                    f = tc_ex2((m - mx) * c2);
                    m = mx;
                    raise = true;
                }
                // c s - r in one rounding leaves c m - r, r's own rounding: far below 1 for the scores of a
                // model, but the exponent of a huge one could overflow.  Those rows subtract first.
                float from = m == -INFINITY ? 0.f : m, ref = from * c2;
                const bool huge = !(fabsf(ref) < 1048576.f);
                if (huge) ref = 0.f;
                else from = 0.f;
                if (__any_sync(0xffffffffu, huge)) {
#pragma unroll
                    for (int u = 0; u < kTcKeys; ++u) s[u] -= from;
                }
                if (__any_sync(0xffffffffu, raise)) {
                    // every product before S(j) is complete: O is free
                    l *= f;
#pragma unroll
                    for (int c = 0; c < DIM; c += 16) {
                        float o[16];
                        umma::tmem_ld16(tO + c, o);
                        umma::tmem_wait_ld();
#pragma unroll
                        for (int u = 0; u < 16; ++u) o[u] *= f;
                        umma::tmem_st16(tO + c, o);
                    }
                }
                const unsigned long long cc = f2pack(c2, c2), rr = f2pack(-ref, -ref), ones = f2pack(1.f, 1.f);
                unsigned long long sum[2] = {0ull, 0ull};
#pragma unroll
                for (int c = 0; c < kTcKeys; c += 32) {
                    uint32_t w[16];
#pragma unroll
                    for (int u = 0; u < 16; ++u) {
                        float e0, e1;
                        f2unpack(f2fma(f2pack(s[c + 2 * u], s[c + 2 * u + 1]), cc, rr), e0, e1);
                        e0 = tc_ex2(e0);
                        e1 = tc_ex2(e1);
                        sum[u & 1] = f2fma(f2pack(e0, e1), ones, sum[u & 1]);
                        w[u] = tc_pack(e0, e1);
                    }
                    umma::tmem_st16(tS + c / 2, *reinterpret_cast<const float(*)[16]>(w));
                }
                {
                    float x0, x1, x2, x3;
                    f2unpack(sum[0], x0, x1);
                    f2unpack(sum[1], x2, x3);
                    l += (x0 + x1) + (x2 + x3);
                }
                if (t == 0 && !sh && x.len < a.own.n && k0 + kTcKeys > x.len) {
                    // rows of V behind the sequence's length may hold anything: 0 x NaN is not 0
                    const unsigned nv = n + 2 * (j - x.j0) + 1;
                    ok = tc_wait(&mbar[Sh::FULL + nv % NST], (nv / NST) & 1, abort_flag);
                    if (!__all_sync(0xffffffffu, ok)) { dead = true; break; }
                    if (r >= x.len - k0) {
#pragma unroll
                        for (int c = 0; c < DIM / 8; ++c)
                            *reinterpret_cast<uint4*>(ring + (nv % NST) * Sh::ST + (c >> 3) * (kTcKeys * 128) + r * 128 +
                                                      (c & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
                    }
                    umma::fence_async_smem();
                }
                umma::tmem_wait_st();
                umma::fence_before_sync();
                umma::mbar_arrive(&mbar[Sh::PFULL + t]);
            }
            if (dead) break;
            n += 2 * (x.j1 - x.j0);
            const bool any = x.j1 > x.j0;
            if (any) {
                const bool ok = tc_wait(&mbar[Sh::OFULL + t], no & 1, abort_flag);
                ++no;
                if (!__all_sync(0xffffffffu, ok)) { dead = true; break; }
                umma::fence_after_sync();
            }
            const float inv = l == 0.f ? 0.f : 1.f / l;
            const float l2 = l == 0.f ? -INFINITY : fmaf(m, c2, log2f(l));
            // The row's place is found again: kept across the loop it would cost registers there.
            int Ro = row_ok ? R : 0;
            asm volatile("" : "+r"(Ro));
            const size_t at = row_at(a, x.n0, x.g, Ro).o;
            const size_t po = (size_t)x.part * a.B * a.T * a.Hq + at;
            uint8_t* to = !row_ok ? nullptr
                          : a.part_o ? reinterpret_cast<uint8_t*>(a.part_o + po * DIM)
                                     : reinterpret_cast<uint8_t*>((bf16*)a.y + at * DIM);
            // Rows leave through shared memory, 64 bytes at a time, so that four lanes write one row's: a
            // thread that wrote its own row would touch 32 lines with every instruction, and the
            // barriers of the next item would wait behind those stores.
            uint8_t* out = smem + Sh::OUT + warp * 2048;
            auto leave = [&](int c, const uint32_t (&w)[16]) {
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    *reinterpret_cast<uint4*>(out + lane * 64 + ((u ^ (lane >> 1 & 3)) << 4)) =
                        make_uint4(w[4 * u], w[4 * u + 1], w[4 * u + 2], w[4 * u + 3]);
                __syncwarp();
#pragma unroll
                for (int it = 0; it < 4; ++it) {
                    const int rr = 8 * it + (lane >> 2), u = lane & 3;
                    const unsigned long long row = __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(to), rr);
                    if (row)
                        *reinterpret_cast<uint4*>(row + 64 * c + 16 * u) =
                            *reinterpret_cast<const uint4*>(out + rr * 64 + ((u ^ (rr >> 1 & 3)) << 4));
                }
                __syncwarp();
            };
#pragma unroll 1
            for (int c = 0; c < DIM / 16; ++c) {
                float o[16];
                uint32_t w[16];
                if (any) {
                    umma::tmem_ld16(tO + 16 * c, o);
                    umma::tmem_wait_ld();
                }
#pragma unroll
                for (int u = 0; u < 16; ++u) o[u] = l == 0.f ? 0.f : o[u] * inv;
                if (a.part_o) {
                    leave(c, *reinterpret_cast<const uint32_t(*)[16]>(o));
                } else {
#pragma unroll
                    for (int u = 0; u < 8; ++u) w[u] = tc_pack(o[2 * u], o[2 * u + 1]);
                    ++c;
                    if (any) {
                        umma::tmem_ld16(tO + 16 * c, o);
                        umma::tmem_wait_ld();
                    }
#pragma unroll
                    for (int u = 0; u < 16; ++u) o[u] = l == 0.f ? 0.f : o[u] * inv;
#pragma unroll
                    for (int u = 0; u < 8; ++u) w[8 + u] = tc_pack(o[2 * u], o[2 * u + 1]);
                    leave(c >> 1, w);
                }
            }
            if (row_ok) {
                if (a.part_o) a.part_l[po] = l2;
                else if (a.lse) a.lse[at] = l2 * 0.6931471805599453f;
            }
        }
    }
    umma::fence_before_sync();
    __syncthreads();
    if (tid == 0 && *abort_flag) atomicOr(&g_attn_err, 1);
    if (warp == 0) umma::tmem_dealloc(tmem, 512);
}

namespace {

// A tensor of keys or values as [batch][head][half][key][64 dims]: one box of 128 keys lands as
// [half][128 keys][128 bytes], swizzled.
bool tc_map(TcArgs& p, int which, const void* base, int d, int n, long long ks, int H, long long kh, int B, long long kb) {
    typedef CUresult (*Encode)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                               const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                               CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
    static const Encode encode = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess)
            return (Encode) nullptr;
        return (Encode)f;
    }();
    if (!encode) return false;
    p.mh[which] = H > 1 && kh > 0;
    p.mb[which] = B > 1 && kb > 0;
    if (!p.mh[which]) { H = 1; kh = 8; }
    if (!p.mb[which]) { B = 1; kb = 8; }
    if (n == 1) ks = 8;
    const cuuint64_t dims[5] = {64, (cuuint64_t)n, (cuuint64_t)(d / 64), (cuuint64_t)H, (cuuint64_t)B};
    const cuuint64_t strides[4] = {(cuuint64_t)ks * 2, 128, (cuuint64_t)kh * 2, (cuuint64_t)kb * 2};
    const cuuint32_t box[5] = {64, kTcKeys, (cuuint32_t)(d / 64), 1, 1}, one[5] = {1, 1, 1, 1, 1};
    return encode(&p.map[which], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void*>(base), dims, strides, box, one,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DIM>
cudaError_t launch_tc_t(const TcArgs& p, int num_sms, cudaStream_t s) {
    using Sh = TcShape<DIM>;
    static std::atomic<unsigned long long> done{0};
    cudaError_t e = allow_smem(attn_tc_kernel<DIM>, Sh::BYTES, &done);
    if (e != cudaSuccess) return e;
    attn_tc_kernel<DIM><<<p.items < num_sms ? p.items : num_sms, kTcThreads, Sh::BYTES, s>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attn_tc(const AttnArgs& a, int num_sms, cudaStream_t s) {
    TcArgs p{};
    const KeySeg &sh = a.shared, &ow = a.own;
    const bool shared = a.by_shared == AttnBy::tiles, own = a.by_own == AttnBy::tiles;
    if (sh.n > 0 && (shared || a.walk) && (!tc_map(p, 0, sh.k, a.d, sh.n, sh.ks, a.Hkv, sh.kh, 1, 0) ||
                                           !tc_map(p, 1, sh.v, a.d, sh.n, sh.vs, a.Hkv, sh.vh, 1, 0)))
        return cudaErrorInvalidValue;
    if (ow.n > 0 && own && (!tc_map(p, 2, ow.k, a.d, ow.n, ow.ks, a.Hkv, ow.kh, a.B, ow.kb) ||
                            !tc_map(p, 3, ow.v, a.d, ow.n, ow.vs, a.Hkv, ow.vh, a.B, ow.vb)))
        return cudaErrorInvalidValue;
    p.a = a;
    const int rows = a.T * a.Gq;
    auto pairs = [](long long n) { return (int)((n + 2 * kTcRows - 1) / (2 * kTcRows)); };
    p.row_tiles[0] = pairs((long long)a.B * rows);
    p.row_tiles[1] = pairs(rows);
    p.parts[0] = shared ? a.parts_shared : 1;
    p.parts[1] = own ? a.parts_own : 1;
    p.chunk[0] = a.chunk_shared / kTcKeys;
    p.chunk[1] = a.chunk_own / kTcKeys;
    p.shared_items = shared ? p.row_tiles[0] * p.parts[0] * a.Hkv : 0;
    p.items = p.shared_items + (own ? p.row_tiles[1] * p.parts[1] * a.Hkv * a.B : 0);
    return a.d == 128 ? launch_tc_t<128>(p, num_sms, s) : launch_tc_t<64>(p, num_sms, s);
}

// Reads and clears this device's error word (waits for the stream).
cudaError_t attn_error_word(int* word, cudaStream_t s) {
    cudaError_t e = cudaMemcpyFromSymbolAsync(word, g_attn_err, sizeof(int), 0, cudaMemcpyDeviceToHost, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    static const int zero = 0;
    if (e == cudaSuccess && *word) e = cudaMemcpyToSymbolAsync(g_attn_err, &zero, sizeof(int), 0, cudaMemcpyHostToDevice, s);
    return e;
}

}  // namespace lola
