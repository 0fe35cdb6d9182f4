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

// The parts of a row put together: with L_p the log2-sum-exp of part p and O_p its
// normalised sum, L = log2 sum 2^L_p and y = sum 2^(L_p - L) O_p.  One warp per row;
// the parts were just written and come from L2.
template <int DIM, typename TOut>
__global__ void __launch_bounds__(128) attn_join_kernel(const __grid_constant__ AttnArgs a) {
    constexpr int EPL = DIM / 32;
    const size_t rows = (size_t)a.B * a.T * a.Hq, row = (size_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (row >= rows) return;
    const int np = a.parts_own + a.parts_shared;
    float m = -INFINITY;
    for (int p = lane; p < np; p += 32) m = fmaxf(m, a.part_l[p * rows + row]);
    m = warp_max(m);
    const float ref = m == -INFINITY ? 0.f : m;
    float sum = 0.f, acc[EPL];
#pragma unroll
    for (int u = 0; u < EPL; ++u) acc[u] = 0.f;
#pragma unroll 4
    for (int p = 0; p < np; ++p) {
        const float w = exp2f(a.part_l[p * rows + row] - ref);
        const float* o = a.part_o + (p * rows + row) * DIM + lane * EPL;
        sum += w;
        if (EPL == 4) {
            const float4 x = *reinterpret_cast<const float4*>(o);
            acc[0] = fmaf(w, x.x, acc[0]); acc[1] = fmaf(w, x.y, acc[1]);
            acc[EPL - 2] = fmaf(w, x.z, acc[EPL - 2]); acc[EPL - 1] = fmaf(w, x.w, acc[EPL - 1]);
        } else {
            const float2 x = *reinterpret_cast<const float2*>(o);
            acc[0] = fmaf(w, x.x, acc[0]); acc[1] = fmaf(w, x.y, acc[1]);
        }
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
    for (int u = 0; u < EPL; ++u) store_as((TOut*)a.y + row * DIM + lane * EPL + u, acc[u] * inv);
    if (a.lse && lane == 0) a.lse[row] = sum == 0.f ? -INFINITY : (ref + log2f(sum)) * 0.6931471805599453f;
}

size_t plan_attn(AttnArgs& a, int num_sms) {
    a.walk = 1;
    a.by_shared = a.by_own = AttnBy::none;
    a.parts_shared = a.parts_own = a.chunk_shared = a.chunk_own = 0;
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
    // Two CTAs per SM of the kernels for few rows, parts of at least 256 keys: four rounds of a CTA;
    // f32 tiles: two per SM, parts of 128 keys; bf16 tiles: one per SM, four tiles of 128 keys.
    auto cut_rows = [&](long long n, long long ctas, int* parts, int* chunk) {
        long long c;
        cut(n, ctas, 2LL * num_sms, 64, f32 ? 128 : 256, parts, &c);
        *chunk = (int)c;
    };
    auto cut_tiles = [&](long long n0, long long n1, long long r, long long heads, int* parts, int* chunk) {
        long long c;
        if (f32) {
            cut(n0 + n1, tiles(r, 64) * heads, 2LL * num_sms, 32, 128, parts, &c);
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
    if (!a.walk) {
        if (all_rows <= few && !f32) {
            a.by_shared = AttnBy::rows;
            cut_rows(P, a.Hkv, &a.parts_shared, &a.chunk_shared);
        } else {
            a.by_shared = AttnBy::tiles;
            cut_tiles(P, 0, all_rows, a.Hkv, &a.parts_shared, &a.chunk_shared);
        }
    }
    if (a.walk || L > 0) {
        const int n0 = a.walk ? P : 0;
        if (rows <= few) {
            a.by_own = AttnBy::rows;
            cut_rows((long long)n0 + L, groups * (f32 ? tiles(rows, 4) : 1), &a.parts_own, &a.chunk_own);
        } else {
            a.by_own = AttnBy::tiles;
            cut_tiles(n0, L, rows, groups, &a.parts_own, &a.chunk_own);
        }
    }
    const int parts = a.parts_own + a.parts_shared;
    if (parts == 1) return 0;
    return (size_t)parts * a.B * a.T * a.Hq * (a.d + 1) * 4;
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
    auto by_tiles = [&](int packed) {
        return f32 ? launch_attn_f32_tiles(a, packed, s) : launch_attn_tc(a, packed, num_sms, s);
    };
    if (a.by_shared == AttnBy::tiles && !run(by_tiles(1))) return e;
    if (a.by_own == AttnBy::tiles && !run(by_tiles(0))) return e;
    if ((a.by_shared == AttnBy::rows || a.by_own == AttnBy::rows) &&
        !run(f32 ? launch_attn_f32_rows(a, s) : launch_attn_rows(a, s)))
        return e;
    if (a.part_o) {
        const unsigned grid = (unsigned)(((size_t)a.B * a.T * a.Hq + 3) / 4);
        if (f32) {
            if (a.d == 128) attn_join_kernel<128, float><<<grid, 128, 0, s>>>(a);
            else attn_join_kernel<64, float><<<grid, 128, 0, s>>>(a);
        } else {
            if (a.d == 128) attn_join_kernel<128, __nv_bfloat16><<<grid, 128, 0, s>>>(a);
            else attn_join_kernel<64, __nv_bfloat16><<<grid, 128, 0, s>>>(a);
        }
        run(cudaGetLastError());
    }
    return e;
}

}  // namespace lola
