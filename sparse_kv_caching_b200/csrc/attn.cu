// Exact attention beside the hybrid layer: how a call is cut into CTAs, and the
// kernel that joins the parts of a row.
//   y = sum_i p_i v_i, p = softmax(scale q.k) over a row's shared keys and its own.
// Every kernel makes one pass over its keys with the running maximum m and sum l
// of the softmax: a tile of scores x moves them to m' = max(m, max x), l' =
// l 2^(m - m') + sum 2^(x - m') (x in the log2 domain) and the accumulator likewise;
// y = acc / l.  A row that reads no key gives y = 0, lse = -inf.
#include "attn.h"
#include "device_common.cuh"

namespace lola {

__device__ __forceinline__ void store_as(float* p, float x) { *p = x; }
__device__ __forceinline__ void store_as(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

// The parts of a row put together: with L_p the log2-sum-exp of part p and O_p its
// normalised sum, L = log2 sum 2^L_p and y = sum 2^(L_p - L) O_p.  One warp per row;
// the parts were just written and come from L2.
template <int DIM, typename TOut>
__global__ void __launch_bounds__(128) attn_join_kernel(const __grid_constant__ AttnArgs a) {
    constexpr int EPL = DIM / 32;
    const size_t rows = (size_t)a.B * a.T * a.Hq, row = (size_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    attn_wait_before();
    if (row >= rows) return;
    // parts in part_o: [p0, p1); of a group whose rounds were dealt evenly and that a cut goes through
    // (k = 0 shared, 1 own): the slots of CTAs c0 .. c1 instead
    int p0 = 0, p1 = a.parts_shared + a.parts_own;
    int total = 0, runs = 0, gb[2] = {0, 0}, c0[2] = {0, 0}, c1[2] = {-1, -1}, rr[2] = {0, 0}, g = 0;
    if (a.even) {
        const int h = (int)(row % a.Hq), n = (int)(row / a.Hq), b = n / a.T;
        g = h / a.Gq;
        const bool own = a.by_own == AttnBy::rows;
        const int sh = a.by_shared == AttnBy::rows ? (a.shared.n + kRwRound - 1) / kRwRound : 0;
        total = sh + (own ? a.goff[a.B] : 0);
        runs = min(a.even, total);
        auto cta = [&](int x) { return (int)(((x + 1LL) * runs - 1) / total); };
        if (sh) {
            c0[0] = 0;
            c1[0] = cta(sh - 1);
            rr[0] = n * a.Gq + h % a.Gq;
            if (c1[0] == 0) c1[0] = -1;
            else p0 = 1;
        }
        if (own) {
            const int o = a.goff[b], len = a.goff[b + 1] - o;
            gb[1] = sh + o;
            c0[1] = cta(gb[1]);
            c1[1] = cta(gb[1] + len - 1);
            rr[1] = (n - b * a.T) * a.Gq + h % a.Gq;
            if (c0[1] == c1[1]) c1[1] = -1;
            else p1 = a.parts_shared;
        }
        if (!a.part_o) {                       // one group a row, shared or own
            if (c1[0] < 0 && c1[1] < 0) return;        // written whole
            p1 = p0;
        }
    }
    // A batch of 32 parts at a time: lane i looks up part i and its weight, then all lanes add its row.
    const int np = p1 - p0, ns0 = c1[0] - c0[0] + 1, n = np + (ns0 > 0 ? ns0 : 0) + (c1[1] < 0 ? 0 : c1[1] - c0[1] + 1);
    auto slot = [&](int k, int c) {
        const bool second = c == c0[k] && (int)((long long)total * c / runs) != gb[k];     // not the group that CTA's run begins in
        return (size_t)(2 * (c * a.Hkv + g) + second) * a.slot_rows + rr[k];
    };
    float m = -INFINITY, sum = 0.f, acc[EPL];
#pragma unroll
    for (int u = 0; u < EPL; ++u) acc[u] = 0.f;
    for (int i0 = 0; i0 < n; i0 += 32) {
        const int i = i0 + lane, cnt = min(32, n - i0);
        const float* from = nullptr;
        float l = -INFINITY;
        if (i < np) {
            const size_t q = (p0 + i) * rows + row;
            from = a.part_o + q * DIM;
            l = a.part_l[q];
        } else if (i < n) {
            const int k = i - np < ns0 ? 0 : 1;
            const size_t q = slot(k, c0[k] + i - np - (k && ns0 > 0 ? ns0 : 0));
            from = a.slot_o + q * DIM;
            l = a.slot_l[q];
        }
        const float mn = fmaxf(m, warp_max(l)), ref = mn == -INFINITY ? 0.f : mn, f = exp2f(m - ref), w = exp2f(l - ref);
        m = mn;
        sum = sum * f + warp_sum(w);
#pragma unroll
        for (int u = 0; u < EPL; ++u) acc[u] *= f;
        for (int j0 = 0; j0 < cnt; j0 += 8) {
            float x[8][EPL];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const unsigned long long po = __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(from), j0 + j);
                const float* row_p = reinterpret_cast<const float*>(po) + lane * EPL;
#pragma unroll
                for (int u = 0; u < EPL; ++u) x[j][u] = 0.f;
                if (j0 + j < cnt) {
                    if (EPL == 4) *reinterpret_cast<float4*>(x[j]) = *reinterpret_cast<const float4*>(row_p);
                    else *reinterpret_cast<float2*>(x[j]) = *reinterpret_cast<const float2*>(row_p);
                }
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float wj = __shfl_sync(0xffffffffu, w, j0 + j);
#pragma unroll
                for (int u = 0; u < EPL; ++u) acc[u] = fmaf(wj, x[j][u], acc[u]);
            }
        }
    }
    const float ref = m == -INFINITY ? 0.f : m;
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
    for (int u = 0; u < EPL; ++u) store_as((TOut*)a.y + row * DIM + lane * EPL + u, acc[u] * inv);
    if (a.lse && lane == 0) a.lse[row] = sum == 0.f ? -INFINITY : (ref + log2f(sum)) * 0.6931471805599453f;
}

size_t plan_attn(AttnArgs& a, int num_sms) {
    a.walk = 1;
    a.by_shared = a.by_own = AttnBy::none;
    a.parts_shared = a.parts_own = a.chunk_shared = a.chunk_own = a.even = a.slot_rows = a.beside = 0;
    const bool f32 = a.dtype == 0;
    const int rows = a.T * a.Gq, P = a.shared.n, L = a.own.n;
    const long long groups = (long long)a.B * a.Hkv, all_rows = (long long)a.B * rows;
    auto tiles = [](long long n, long long of) { return (n + of - 1) / of; };
    // n keys (or key tiles) cut into parts of a multiple of `unit` for each of `ctas` CTAs, as many as
    // `slots` CTAs run at once, of at least `least`
    auto cut = [&](long long n, long long ctas, long long slots, int unit, int least, int* parts, long long* chunk) {
        long long k = slots / ctas;
        if (k > n / least) k = n / least;
        if (k < 1) k = 1;
        *chunk = tiles(tiles(n, k), unit) * unit;
        if (*chunk == 0) *chunk = unit;
        *parts = n > 0 ? (int)tiles(n, *chunk) : 1;
    };
    // f32: parts of at least 128 keys, four CTAs per SM (two at a time: ragged lengths even out); bf16: one
    // CTA per SM, parts of at least four tiles of 128 keys.
    auto cut_tiles = [&](long long n0, long long n1, long long r, long long heads, int* parts, int* chunk) {
        long long c;
        if (f32) {
            cut(n0 + n1, tiles(r, 64) * heads, 4LL * num_sms, 64, 128, parts, &c);
            *chunk = (int)c;
        } else {
            cut(tiles(n0, 128) + tiles(n1, 128), tiles(r, 256) * heads, num_sms, 1, 4, parts, &c);
            *chunk = (int)(c * 128);
        }
    };
    const int few = f32 ? kF32RowsMax : kRowsMax;
    // The shared keys once for the whole batch, or again for each sequence (from L2)?  Together, a
    // row needs no join.
    if (a.B > 1 && P > 0) {
        if (f32) {
            // seconds: re-reading 8 d bytes a key for every four rows at 8 TB/s against 64-row tiles of
            // 2 d multiply-adds at 25 T/s, and about 4 us of another kernel and the join
            const double each = (double)P * a.Hkv * a.d * 1e-12;
            const double again = rows <= few ? (double)a.B * tiles(rows, 4) : 5.0 * a.B * tiles(rows, 64);
            a.walk = (again - 5.0 * tiles(all_rows, 64)) * each < 4e-6;
        } else if (P > 512) {
            const int of = all_rows <= few ? few : 128;
            a.walk = a.B * tiles(rows, of) < 2 * tiles(all_rows, of);
        }
    }
    const int n0 = a.walk ? P : 0;              // shared keys that a sequence's rows read before their own
    if (!a.walk) {
        if (all_rows <= few && !f32) {
            a.by_shared = AttnBy::rows;
            a.parts_shared = 1;
        } else {
            a.by_shared = AttnBy::tiles;
            cut_tiles(P, 0, all_rows, a.Hkv, &a.parts_shared, &a.chunk_shared);
        }
    }
    if (a.walk || L > 0) {
        if (rows > few) {
            a.by_own = AttnBy::tiles;
            cut_tiles(n0, L, rows, groups, &a.parts_own, &a.chunk_own);
        } else {
            a.by_own = AttnBy::rows;
            a.parts_own = 1;
            if (f32) {
                // (two CTAs per SM: with four the join of twice the parts costs more than the shorter walks
                // save, 20 against 15 us for 7 tokens after 4095 shared keys)
                long long c;
                cut((long long)n0 + L, groups * tiles(rows, 4), 2LL * num_sms, 32, 64, &a.parts_own, &c);
                a.chunk_own = (int)c;
            }
        }
    }
    if (!f32 && (a.by_own == AttnBy::rows || a.by_shared == AttnBy::rows)) {
        // The shared keys' tiles are bound by the tensor cores and by their own begin and end, the own keys
        // by HBM, or by how fast an SM turns them over: they run at the same time on SMs of their own, in
        // the shares that end together.  Measured (32 / 8 heads, d 128), in us: 1.75 for each pair of row
        // tiles and key tile and 20 for the rest; 0.04 MB per us and SM, 5.2 in all, and 5 for the rest.
        long long slots = 2LL * num_sms;
        const long long base = tiles(all_rows, 256) * a.Hkv;
        if (a.by_shared == AttnBy::tiles && a.by_own == AttnBy::rows && base + a.Hkv / 2 < num_sms) {
            const long long key_tiles = tiles(P, 128);
            const double mb = (double)groups * L * 4 * a.d * 1e-6;
            double best = 1e30;
            for (long long k = 1; base * k + a.Hkv / 2 < num_sms; ++k) {
                const long long chunk = tiles(key_tiles, k), rest = num_sms - base * tiles(key_tiles, chunk);
                const double t_own = 5 + mb / (0.04 * rest < 5.2 ? 0.04 * rest : 5.2), t_shared = 20 + 1.75 * chunk;
                const double t = t_own > t_shared ? t_own : t_shared;
                if (t < best) {
                    best = t;
                    a.parts_shared = (int)tiles(key_tiles, chunk);
                    a.chunk_shared = (int)(chunk * 128);
                    slots = 2 * rest;
                }
            }
            a.beside = 1;
        }
        // Rounds of 64 keys, a CTA per group or dealt evenly?  In rounds: a CTA on an SM of its own or with
        // one neighbour takes about one unit of time for each, and four for its begin and end; evenly
        // dealt work needs the join, about four more.
        const long long sh = a.by_shared == AttnBy::rows ? tiles(P, kRwRound) : 0;
        const long long own = a.by_own == AttnBy::rows ? tiles((long long)n0 + L, kRwRound) : 0;
        const long long ctas = (sh ? a.Hkv : 0) + (own ? groups : 0), all = sh + own * a.B;      // of one head
        const long long most = sh > own ? sh : own, runs = slots / a.Hkv < all ? slots / a.Hkv : all;
        if (runs > 0 && all < (1LL << 30) && tiles(all, runs) + 8 < tiles(ctas, slots) * (most + 4)) a.even = (int)runs;
        a.slot_rows = (int)(sh ? all_rows : rows);
    }
    const int parts = a.parts_own + a.parts_shared;
    size_t bytes = 0;
    auto take = [&](size_t n) { bytes += (n + 255) & ~(size_t)255; };
    if (parts > 1) take((size_t)parts * a.B * a.T * a.Hq * (a.d + 1) * 4);
    if (a.even) {
        take((size_t)2 * a.even * a.Hkv * a.slot_rows * (a.d + 1) * 4);
        take(((size_t)a.B + 1) * 4);
    }
    return bytes;
}

void place_attn(AttnArgs& a, void* workspace) {
    char* w = (char*)workspace;
    const int parts = a.parts_own + a.parts_shared;
    auto take = [&](size_t n) { char* p = w; w += (n + 255) & ~(size_t)255; return p; };
    if (parts > 1) {
        const size_t rows = (size_t)parts * a.B * a.T * a.Hq;
        a.part_o = (float*)take(rows * (a.d + 1) * 4);
        a.part_l = a.part_o + rows * a.d;
    }
    if (a.even) {
        const size_t rows = (size_t)2 * a.even * a.Hkv * a.slot_rows;
        a.slot_o = (float*)take(rows * (a.d + 1) * 4);
        a.slot_l = a.slot_o + rows * a.d;
        a.goff = (int*)take(((size_t)a.B + 1) * 4);
    }
}

cudaError_t launch_attn(const AttnArgs& a, int num_sms, int* launches, cudaStream_t s) {
    *launches = 0;
    cudaError_t e = cudaSuccess;
    auto run = [&](cudaError_t x) {
        e = x;
        ++*launches;
        return x == cudaSuccess;
    };
    const bool f32 = a.dtype == 0;
    if (f32) {
        if (a.by_shared == AttnBy::tiles && !run(launch_attn_f32_tiles(a, 1, s))) return e;
        if (a.by_own == AttnBy::tiles && !run(launch_attn_f32_tiles(a, 0, s))) return e;
    } else if ((a.by_shared == AttnBy::tiles || a.by_own == AttnBy::tiles) && !run(launch_attn_tc(a, num_sms, s))) {
        return e;
    }
    if ((a.by_shared == AttnBy::rows || a.by_own == AttnBy::rows) &&
        !run(f32 ? launch_attn_f32_rows(a, s) : launch_attn_rows(a, s)))
        return e;
    if (a.part_o || a.even) {
        const unsigned grid = (unsigned)(((size_t)a.B * a.T * a.Hq + 3) / 4);
        auto join = f32 ? (a.d == 128 ? attn_join_kernel<128, float> : attn_join_kernel<64, float>)
                        : (a.d == 128 ? attn_join_kernel<128, __nv_bfloat16> : attn_join_kernel<64, __nv_bfloat16>);
        run(attn_launch(join, grid, 128, 0, true, s, a));
    }
    return e;
}

}  // namespace lola
