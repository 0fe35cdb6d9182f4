// Exact attention for few rows per kv head (decode steps, short drafts), bf16.
//
// A group's R <= 16 rows (queries x heads of the kv group) read N keys: 4 R d N
// operations on 4 d N bytes, R operations a byte, so the kernel is bound by HBM
// as long as each key is read once for all its rows and enough loads are in
// flight.  Keys go by rounds of 64, 16 for each of a CTA's four warps: a warp copies
// its 16 K and V rows into its own ring of stages with cp.async two rounds ahead
// and waits for no other warp; S = Q K^T and O += P V run on the warp-level tensor
// instructions (m16n8k16: a 16-row tile of Q in registers, which a tile of 128 rows
// on the SM-level unit would leave almost empty).  Softmax: running maximum and
// sum per row and warp, f32; the accumulator is rescaled only when a maximum
// rises.  P is fed as two bf16 parts (its rounding and the remainder): the second
// product is free under the loads and keeps the weights to 2^-16.
//
// How the rounds are dealt (plan_attn).  Whole: a CTA per group, which then writes y
// itself.  Even: for each kv head the rounds of all its groups in one list, cut into
// equal runs for two CTAs per SM, whatever the sequences' lengths; the copies of a run
// do not stop where one group ends and the next begins.  The heads' lists are cut
// alike and their CTAs start together, so that the rows of one token, which lie next to
// each other, are read at about the same time.  A group that lies inside a run is written
// whole; what a CTA has of a group that a cut goes through is left in one of its two slots
// (the group its run begins in, the one it ends in), and attn_join_kernel puts the
// slots together.
// B200, one token of 64 sequences against 1500 states, 32/8 heads, d 128: 64.9 us for 393 MB,
// 6.07 TB/s (93 % of a copy); a CTA per group took 70 us for ragged lengths, dealt evenly 56.
#include "attn.h"
#include "umma.cuh"

namespace lola {

constexpr int kRwWarps = 4, kRwKeys = 16, kRwStages = 3;
static_assert(kRwRound == kRwWarps * kRwKeys, "a round");

__device__ __forceinline__ void rw_ldsm(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
__device__ __forceinline__ void rw_ldsm_t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
__device__ __forceinline__ void rw_mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float rw_ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t rw_pack(float lo, float hi) {
    __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&v);
}
// x = hi + lo in bf16 parts
__device__ __forceinline__ void rw_split(float x0, float x1, uint32_t& hi, uint32_t& lo) {
    hi = rw_pack(x0, x1);
    lo = rw_pack(x0 - __uint_as_float(hi << 16), x1 - __uint_as_float(hi & 0xFFFF0000u));
}

template <int DIM>
struct RowsShape {
    static constexpr int STAGE = 2 * kRwKeys * DIM * 2;               // K rows, then V rows
    static constexpr int WARP = kRwStages * STAGE;
    static constexpr int RED = kRwWarps * WARP;                       // 8 rows of every warp's O where a group ends
    static constexpr int ML = RED + kRwWarps * 8 * DIM * 4, SCAN = ML + kRwWarps * 8 * 8, BYTES = SCAN + 64;
};

// A place in a kv head's list of rounds: first the shared keys' group (where this kernel reads
// them apart), then each sequence's.
struct RowsAt {
    int shared, b, round, rounds;
};

__device__ __forceinline__ int rw_rounds(const AttnArgs& a, int b) {  // of one group of sequence b
    return max(1, (int)(((a.walk ? a.shared.n : 0) + (long long)own_length(a, b) + kRwRound - 1) / kRwRound));
}
__device__ __forceinline__ void rw_next(const AttnArgs& a, RowsAt& x) {
    if (++x.round < x.rounds) return;
    x.round = 0;
    x.b = x.shared ? 0 : x.b + 1;
    x.shared = 0;
    if (x.b < a.B) x.rounds = rw_rounds(a, x.b);
}

template <int DIM>
__global__ void __launch_bounds__(kRwWarps * 32, 2) attn_rows_kernel(const __grid_constant__ AttnArgs a) {
    using Sh = RowsShape<DIM>;
    using bf16 = __nv_bfloat16;
    constexpr int KC = DIM / 8;                 // 16-byte chunks of a key row
    constexpr int RB = DIM * 2;                 // its bytes
    extern __shared__ __align__(128) uint8_t smem[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = blockIdx.x % a.Hkv, run = blockIdx.x / a.Hkv;
    attn_let_next_begin();

    // ---- this CTA's run of rounds ----
    RowsAt at{};                                // where it begins
    int left;                                   // rounds
    const int sh_rounds = a.by_shared == AttnBy::rows ? (a.shared.n + kRwRound - 1) / kRwRound : 0;
    if (!a.even) {
        at.shared = sh_rounds && run == 0;
        at.b = at.shared ? 0 : run - (sh_rounds ? 1 : 0);
        at.rounds = at.shared ? sh_rounds : rw_rounds(a, at.b);
        left = at.rounds;
    } else {
        // rounds before each sequence (goff): every CTA sums them, the first one leaves them for the join
        int* scan = reinterpret_cast<int*>(smem + Sh::SCAN);
        const int own = a.by_own == AttnBy::rows, nb = own ? a.B : 0;
        const int per = (nb + kRwWarps * 32 - 1) / (kRwWarps * 32), b0 = min(nb, tid * per), b1 = min(nb, b0 + per);
        int mine = 0;
        for (int b = b0; b < b1; ++b) mine += rw_rounds(a, b);
        int incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
        }
        if (lane == 31) scan[warp] = incl;
        __syncthreads();
        int before = incl - mine, all = 0;
        for (int w = 0; w < kRwWarps; ++w) {
            if (w < warp) before += scan[w];
            all += scan[w];
        }
        const int total = sh_rounds + all, runs = min(a.even, total), c = min(run, runs);
        const int begin = (int)((long long)total * c / runs), end = (int)((long long)total * min(c + 1, runs) / runs);
        left = end - begin;
        if (blockIdx.x == 0) {
            int o = before;
            for (int b = b0; b < b1; ++b) {
                a.goff[b] = o;
                o += rw_rounds(a, b);
            }
            if (tid == 0) a.goff[a.B] = all;
        }
        if (begin >= sh_rounds) {
            const int x = begin - sh_rounds;
            int o = before;
            for (int b = b0; b < b1; ++b) {
                const int n = rw_rounds(a, b);
                if (x >= o && x < o + n) {
                    scan[8] = b;
                    scan[9] = x - o;
                    scan[10] = n;
                }
                o += n;
            }
        }
        __syncthreads();
        if (begin < sh_rounds) at = {1, 0, begin, sh_rounds};
        else at = {0, scan[8], scan[9], scan[10]};
    }
    if (left == 0) {
        if (a.beside) attn_wait_before();
        return;
    }

    // ---- copies, two rounds ahead of the products ----
    uint8_t* ring = smem + warp * Sh::WARP;
    RowsAt ahead = at;
    int to_fetch = left;
    int stage_in = 0;
    const bf16 *fk = nullptr, *fv = nullptr;    // this lane's chunk of key 0 of the group, shared or own
    const bf16 *sk = nullptr, *sv = nullptr;    // ... of the shared keys, in front of the own ones (walk)
    int np0 = 0, n_keys = 0;
    long long fks = 0, fvs = 0;
    auto enter = [&] {                          // pointers of the group `ahead` is in
        const int c = 8 * (lane % KC);
        const KeySeg& sg = ahead.shared ? a.shared : a.own;
        fk = (const bf16*)sg.k + ahead.b * sg.kb + (long long)g * sg.kh + c;
        fv = (const bf16*)sg.v + ahead.b * sg.vb + (long long)g * sg.vh + c;
        fks = sg.ks;
        fvs = sg.vs;
        np0 = !ahead.shared && a.walk ? a.shared.n : 0;
        if (np0) {
            sk = (const bf16*)a.shared.k + (long long)g * a.shared.kh + c;
            sv = (const bf16*)a.shared.v + (long long)g * a.shared.vh + c;
        }
        n_keys = ahead.shared ? a.shared.n : np0 + own_length(a, ahead.b);
    };
    enter();
    auto fetch = [&] {
        if (to_fetch > 0) {
            uint8_t* st = ring + stage_in * Sh::STAGE;
            const int k0 = ahead.round * kRwRound + warp * kRwKeys;
            constexpr int RPI = 32 / KC;        // rows per pass
            const int c = lane % KC;
            auto copy = [&](int r, const bf16* kp, const bf16* vp, bool ok) {
                const uint32_t off = r * RB + ((c ^ (r & 7)) << 4);
                umma::cp_async16_zfill(st + off, ok ? (const void*)kp : a.q, ok);
                umma::cp_async16_zfill(st + kRwKeys * RB + off, ok ? (const void*)vp : a.q, ok);
            };
            if (k0 >= np0 || k0 + kRwKeys <= np0) {       // all own (or the shared group's), or all shared
                const bool front = k0 < np0;
                const long long ks = front ? a.shared.ks : fks, vs = front ? a.shared.vs : fvs;
                const int key = k0 + lane / KC;
                const bf16* kp = (front ? sk : fk) + (key - (front ? 0 : np0)) * ks;
                const bf16* vp = (front ? sv : fv) + (key - (front ? 0 : np0)) * vs;
#pragma unroll
                for (int it = 0; it < kRwKeys / RPI; ++it) {
                    copy(it * RPI + lane / KC, kp, vp, key + it * RPI < n_keys);
                    kp += RPI * ks;
                    vp += RPI * vs;
                }
            } else {
#pragma unroll 1
                for (int it = 0; it < kRwKeys / RPI; ++it) {
                    const int r = it * RPI + lane / KC, key = k0 + r;
                    const bool front = key < np0;
                    copy(r, front ? sk + key * a.shared.ks : fk + (key - np0) * fks,
                         front ? sv + key * a.shared.vs : fv + (key - np0) * fvs, key < n_keys);
                }
            }
            stage_in = stage_in + 1 == kRwStages ? 0 : stage_in + 1;
            const bool last = ahead.round + 1 == ahead.rounds;
            rw_next(a, ahead);
            if (--to_fetch > 0 && last) enter();
        }
        umma::cp_async_commit();
    };
#pragma unroll
    for (int j = 0; j < kRwStages - 1; ++j) fetch();

    // ---- queries: A fragments (row lane/4 and + 8, dims 2 (lane%4) and + 8) ----
    uint32_t qf[DIM / 16][4];
    int lim[2];                                 // keys of the group that each of this lane's rows reads
    int R = 0, n0 = 0;
    auto queries = [&](const RowsAt& x) {
        n0 = x.shared ? 0 : x.b * a.T;
        R = (x.shared ? a.B : 1) * a.T * a.Gq;
        const int len = x.shared ? 0 : own_length(a, x.b), ns = x.shared || a.walk ? a.shared.n : 0;
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
            const int r = hh * 8 + lane / 4;
            const bool ok = r < R;
            const RowAt y = row_at(a, n0, g, ok ? r : 0);
            const uint32_t* qp = reinterpret_cast<const uint32_t*>((const bf16*)a.q + y.q) + lane % 4;
            lim[hh] = ns + (x.shared ? 0 : own_visible(a, len, y.t));
#pragma unroll
            for (int kk = 0; kk < DIM / 16; ++kk) {
                qf[kk][hh] = ok ? qp[8 * kk] : 0u;
                qf[kk][hh + 2] = ok ? qp[8 * kk + 4] : 0u;
            }
        }
    };
    queries(at);

    float o[DIM / 8][4], m[2], l[2];
    auto clear = [&] {
#pragma unroll
        for (int n = 0; n < DIM / 8; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[n][i] = 0.f;
        m[0] = m[1] = -INFINITY;
        l[0] = l[1] = 0.f;
    };
    clear();
    const uint32_t ring_s = umma::smem_addr(ring);
    // ldmatrix addresses: lane i gives row (i % 8) of 8 x 8 matrix i / 8
    const int krow = (lane & 7) + ((lane >> 4) << 3), kch = (lane >> 3) & 1;      // K: matrices (keys, dims) 00 01 10 11
    const int vrow = (lane & 7) + (((lane >> 3) & 1) << 3), vch = lane >> 4;      // V: (keys, dims) 00 10 01 11
    int stage = 0, from = at.round;             // `from`: this CTA's first round of the group
    bool first_group = true;
    for (; left > 0; --left) {
        umma::cp_async_wait<kRwStages - 2>();
        __syncwarp();
        fetch();                                // into the stage read one round ago
        const uint32_t ks = ring_s + stage * Sh::STAGE, vs = ks + kRwKeys * RB;
        stage = stage + 1 == kRwStages ? 0 : stage + 1;
        const int k0 = at.round * kRwRound + warp * kRwKeys;
        // (loads of four steps in front of their products, two accumulators for each 8 keys: the warp has one
        // neighbour on its scheduler at most, so latencies show)
        float s2[2][2][4];
#pragma unroll
        for (int i = 0; i < 16; ++i) s2[i >> 3][i >> 2 & 1][i & 3] = 0.f;
#pragma unroll
        for (int k4 = 0; k4 < DIM / 16; k4 += 4) {
            uint32_t kf[4][4];
#pragma unroll
            for (int k = 0; k < 4; ++k) rw_ldsm(kf[k], ks + krow * RB + (((2 * (k4 + k) + kch) ^ (krow & 7)) << 4));
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                rw_mma(s2[k & 1][0], qf[k4 + k], kf[k][0], kf[k][1]);
                rw_mma(s2[k & 1][1], qf[k4 + k], kf[k][2], kf[k][3]);
            }
        }
        float s[2][4];
#pragma unroll
        for (int i = 0; i < 8; ++i) s[i >> 2][i & 3] = s2[0][i >> 2][i & 3] + s2[1][i >> 2][i & 3];
        uint32_t ph[4], pl[4];
        float f[2];
        bool up = false;
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
            // this lane's keys: 2 (lane % 4) + {0, 1} of each 8-key tile
            float x[4], mx = -INFINITY;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int key = k0 + (i >> 1) * 8 + 2 * (lane & 3) + (i & 1);
                x[i] = key < lim[hh] ? s[i >> 1][2 * hh + (i & 1)] * a.scale_log2 : -INFINITY;
                mx = fmaxf(mx, x[i]);
            }
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            const float mn = fmaxf(m[hh], mx), ref = mn == -INFINITY ? 0.f : mn;
            f[hh] = rw_ex2(m[hh] - ref);
            up |= mn != m[hh];
            m[hh] = mn;
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[i] = rw_ex2(x[i] - ref);
                sum += x[i];
            }
            l[hh] = l[hh] * f[hh] + sum;                  // this lane's keys only: summed over lanes at the end
            rw_split(x[0], x[1], ph[hh], pl[hh]);         // A fragment: keys 2 (lane%4), then + 8
            rw_split(x[2], x[3], ph[hh + 2], pl[hh + 2]);
        }
        if (__any_sync(0xffffffffu, up)) {
#pragma unroll
            for (int n = 0; n < DIM / 8; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[n][i] *= f[i >> 1];
        }
#pragma unroll
        for (int n4 = 0; n4 < DIM / 16; n4 += 4) {
            uint32_t vf[4][4];
#pragma unroll
            for (int n = 0; n < 4; ++n) rw_ldsm_t(vf[n], vs + vrow * RB + (((2 * (n4 + n) + vch) ^ (vrow & 7)) << 4));
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    rw_mma(o[2 * (n4 + n)], h ? pl : ph, vf[n][0], vf[n][1]);
                    rw_mma(o[2 * (n4 + n) + 1], h ? pl : ph, vf[n][2], vf[n][3]);
                }
        }
        const bool group_ends = at.round + 1 == at.rounds;
        if (!group_ends && left > 1) {
            ++at.round;
            continue;
        }

        // ---- the group, or the run, ends: the warps' sums meet, 8 rows at a time ----
        const RowsAt done = at;
        const int R_done = R, n0_done = n0;
        rw_next(a, at);
        if (left > 1) queries(at);              // (their loads fly while the sums meet)
        const bool whole = from == 0 && group_ends;
        const size_t rows_all = (size_t)a.B * a.T * a.Hq;
        const int part = done.shared ? 0 : a.parts_shared, slot = 2 * (int)blockIdx.x + (first_group ? 0 : 1);
        float* red = reinterpret_cast<float*>(smem + Sh::RED);
        float2* ml = reinterpret_cast<float2*>(smem + Sh::ML);
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
            const int r0 = hh * 8;
            if (r0 >= R_done) break;
            float x = l[hh];
            x += __shfl_xor_sync(0xffffffffu, x, 1);
            x += __shfl_xor_sync(0xffffffffu, x, 2);
            if ((lane & 3) == 0) ml[warp * 8 + lane / 4] = make_float2(m[hh], x);
            if (r0 + lane / 4 < R_done) {
#pragma unroll
                for (int n = 0; n < DIM / 8; ++n)
                    *reinterpret_cast<float2*>(red + (warp * 8 + lane / 4) * DIM + 8 * n + 2 * (lane & 3)) =
                        make_float2(o[n][2 * hh], o[n][2 * hh + 1]);
            }
            __syncthreads();
            for (int i = tid; i < min(8, R_done - r0) * (DIM / 4); i += kRwWarps * 32) {
                const int r = i / (DIM / 4), c = i % (DIM / 4) * 4;
                float mx = -INFINITY;
#pragma unroll
                for (int w = 0; w < kRwWarps; ++w) mx = fmaxf(mx, ml[w * 8 + r].x);
                const float ref = mx == -INFINITY ? 0.f : mx;
                float sum = 0.f;
                float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int w = 0; w < kRwWarps; ++w) {
                    const float2 z = ml[w * 8 + r];
                    const float f = rw_ex2(z.x - ref);
                    const float4 v = *reinterpret_cast<const float4*>(red + (w * 8 + r) * DIM + c);
                    sum = fmaf(z.y, f, sum);
                    y.x = fmaf(v.x, f, y.x); y.y = fmaf(v.y, f, y.y); y.z = fmaf(v.z, f, y.z); y.w = fmaf(v.w, f, y.w);
                }
                const float inv = sum == 0.f ? 0.f : 1.f / sum;
                y.x *= inv; y.y *= inv; y.z *= inv; y.w *= inv;
                const float l2 = sum == 0.f ? -INFINITY : ref + log2f(sum);
                const size_t at_y = row_at(a, n0_done, g, r0 + r).o;
                if (!whole) {
                    const size_t q = (size_t)slot * a.slot_rows + r0 + r;
                    *reinterpret_cast<float4*>(a.slot_o + q * DIM + c) = y;
                    if (c == 0) a.slot_l[q] = l2;
                } else if (a.part_o) {
                    *reinterpret_cast<float4*>(a.part_o + (part * rows_all + at_y) * DIM + c) = y;
                    if (c == 0) a.part_l[part * rows_all + at_y] = l2;
                } else {
                    *reinterpret_cast<uint2*>((bf16*)a.y + at_y * DIM + c) = make_uint2(rw_pack(y.x, y.y), rw_pack(y.z, y.w));
                    if (a.lse && c == 0) a.lse[at_y] = l2 * 0.6931471805599453f;
                }
            }
            __syncthreads();
        }
        clear();
        first_group = false;
        from = 0;
    }
    umma::cp_async_wait<0>();
    // The tile kernel that runs beside this one writes other parts: with this wait its end comes before this
    // kernel's end, which is what the join waits for.
    if (a.beside) attn_wait_before();
}

template <int DIM>
static cudaError_t launch_rows_t(const AttnArgs& a, cudaStream_t s) {
    using Sh = RowsShape<DIM>;
    static std::atomic<unsigned long long> done{0};
    cudaError_t e = allow_smem(attn_rows_kernel<DIM>, Sh::BYTES, &done);
    if (e != cudaSuccess) return e;
    const int per_head = a.even ? a.even : (a.by_shared == AttnBy::rows) + (a.by_own == AttnBy::rows ? a.B : 0);
    return attn_launch(attn_rows_kernel<DIM>, (unsigned)per_head * a.Hkv, kRwWarps * 32, Sh::BYTES, a.beside != 0, s, a);
}

cudaError_t launch_attn_rows(const AttnArgs& a, cudaStream_t s) {
    return a.d == 128 ? launch_rows_t<128>(a, s) : launch_rows_t<64>(a, s);
}

}  // namespace lola
