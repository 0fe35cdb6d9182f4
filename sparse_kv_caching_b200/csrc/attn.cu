// Exact attention, any shape: y = sum_i p_i v_i, p = softmax(scale q.k) over a
// row's shared keys and its sequence's own keys.  One pass over the keys with
// the running maximum m and sum l of the softmax: a tile of scores x moves
// them to m' = max(m, max x), l' = l e^(m - m') + sum e^(x - m'), and the
// accumulator likewise; y = acc / l, lse = m + log l.  A row that reads no key
// gives y = 0, lse = -inf.  FP32 arithmetic.
#include "attn.h"
#include "device_common.cuh"

namespace lola {

constexpr int kAtRows = 16, kAtKeys = 32, kAtWarps = 8;

template <int DIM, typename TIn>
__global__ void __launch_bounds__(256) attn_kernel(const __grid_constant__ AttnArgs a) {
    constexpr int LD = DIM + 4, CPL = DIM / 32, RPW = kAtRows / kAtWarps;
    __shared__ float qs[kAtRows][DIM];
    __shared__ float ks[kAtKeys][LD];
    __shared__ float vs[kAtKeys][DIM];
    const int g = blockIdx.y, b = blockIdx.z, rows = a.T * a.Gq;
    const int r0 = blockIdx.x * kAtRows, nr = min(kAtRows, rows - r0);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int i = tid; i < kAtRows * DIM / 4; i += 256) {
        const int r = i / (DIM / 4), c = i % (DIM / 4) * 4;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r < nr) {
            const int t = (r0 + r) / a.Gq, h = (r0 + r) % a.Gq;
            x = load4((const TIn*)a.q + b * a.qb + t * a.qs + (long long)(g * a.Gq + h) * a.qh + c);
        }
        *reinterpret_cast<float4*>(&qs[r][c]) = x;
    }
    float m[RPW], l[RPW], acc[RPW][CPL];
#pragma unroll
    for (int i = 0; i < RPW; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.f;
#pragma unroll
        for (int u = 0; u < CPL; ++u) acc[i][u] = 0.f;
    }
    const int len = a.own_len ? min(max(a.own_len[b], 0), a.own.n) : a.own.n;
    for (int seg = 0; seg < 2; ++seg) {
        const KeySeg& sg = seg ? a.own : a.shared;
        const int n = seg ? len : sg.n;
        const TIn* kp = (const TIn*)sg.k + b * sg.kb + g * sg.kh;
        const TIn* vp = (const TIn*)sg.v + b * sg.vb + g * sg.vh;
        for (int k0 = 0; k0 < n; k0 += kAtKeys) {
            __syncthreads();
            for (int i = tid; i < kAtKeys * DIM / 4; i += 256) {
                const int r = i / (DIM / 4), c = i % (DIM / 4) * 4;
                float4 x = make_float4(0.f, 0.f, 0.f, 0.f), z = x;
                if (k0 + r < n) {
                    x = load4(kp + (k0 + r) * sg.ks + c);
                    z = load4(vp + (k0 + r) * sg.vs + c);
                }
                *reinterpret_cast<float4*>(&ks[r][c]) = x;
                *reinterpret_cast<float4*>(&vs[r][c]) = z;
            }
            __syncthreads();
#pragma unroll
            for (int i = 0; i < RPW; ++i) {
                const int r = warp * RPW + i;
                if (r >= nr) break;
                const int t = (r0 + r) / a.Gq;
                const int lim = seg && a.causal ? min(n, len - a.T + t + 1) : n;
                float x = 0.f;
                for (int c = 0; c < DIM; c += 4) {
                    const float4 u = *reinterpret_cast<const float4*>(&qs[r][c]);
                    const float4 w = *reinterpret_cast<const float4*>(&ks[lane][c]);
                    x = fmaf(u.x, w.x, fmaf(u.y, w.y, fmaf(u.z, w.z, fmaf(u.w, w.w, x))));
                }
                x = k0 + lane < lim ? x * a.scale_log2 : -INFINITY;
                const float mn = fmaxf(m[i], warp_max(x)), ref = mn == -INFINITY ? 0.f : mn;
                const float p = k0 + lane < lim ? exp2f(x - ref) : 0.f, f = exp2f(m[i] - ref);
                m[i] = mn;
                l[i] = l[i] * f + warp_sum(p);
#pragma unroll
                for (int u = 0; u < CPL; ++u) acc[i][u] *= f;
                for (int j = 0; j < min(kAtKeys, lim - k0); ++j) {
                    const float pj = __shfl_sync(0xffffffffu, p, j);
#pragma unroll
                    for (int u = 0; u < CPL; ++u) acc[i][u] = fmaf(pj, vs[j][lane + 32 * u], acc[i][u]);
                }
            }
        }
    }
#pragma unroll
    for (int i = 0; i < RPW; ++i) {
        const int r = warp * RPW + i;
        if (r >= nr) break;
        const int t = (r0 + r) / a.Gq, h = g * a.Gq + (r0 + r) % a.Gq;
        const size_t o = ((size_t)b * a.T + t) * a.Hq + h;
        const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];
#pragma unroll
        for (int u = 0; u < CPL; ++u) store_as((TIn*)a.y + o * DIM + lane + 32 * u, acc[i][u] * inv);
        if (a.lse && lane == 0) a.lse[o] = l[i] == 0.f ? -INFINITY : (m[i] + log2f(l[i])) * 0.6931471805599453f;
    }
}

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
    const int rows = a.T * a.Gq, P = a.shared.n, L = a.own.n;
    const long long groups = (long long)a.B * a.Hkv, all_rows = (long long)a.B * rows;
    auto tiles = [](long long n, long long of) { return (n + of - 1) / of; };
    // Few rows: two CTAs per SM, parts of at least 256 keys (four rounds of a CTA).  Tiles: one
    // CTA per SM, parts of at least four key tiles.
    auto cut_rows = [&](long long n, long long ctas, int* parts, int* chunk) {
        long long k = 2LL * num_sms / ctas;
        if (k > n / 256) k = n / 256;
        if (k < 1) k = 1;
        *chunk = (int)(tiles(tiles(n, k), 64) * 64);
        if (*chunk == 0) *chunk = 64;
        *parts = n > 0 ? (int)tiles(n, *chunk) : 1;
    };
    auto cut_tiles = [&](long long n, long long ctas, int* parts, int* chunk) {
        long long k = num_sms / ctas;
        if (k > n / 4) k = n / 4;
        if (k < 1) k = 1;
        const long long c = tiles(n, k) > 0 ? tiles(n, k) : 1;
        *chunk = (int)(c * 128);
        *parts = n > 0 ? (int)tiles(n, c) : 1;
    };
    if (a.dtype != 1) {
        a.by_own = AttnBy::simple;
        a.parts_own = 1;
        return 0;
    }
    // The shared keys once for the whole batch, or again for each sequence (from L2)?  Apart,
    // when that saves row tiles; together, a row needs no join.
    if (a.B > 1 && P > 512) {
        const int of = all_rows <= kRowsMax ? kRowsMax : 128;
        a.walk = a.B * tiles(rows, of) < 2 * tiles(all_rows, of);
    }
    if (!a.walk) {
        if (all_rows <= kRowsMax) {
            a.by_shared = AttnBy::rows;
            cut_rows(P, a.Hkv, &a.parts_shared, &a.chunk_shared);
        } else {
            a.by_shared = AttnBy::tiles;
            cut_tiles(tiles(P, 128), tiles(all_rows, 256) * a.Hkv, &a.parts_shared, &a.chunk_shared);
        }
    }
    if (a.walk || L > 0) {
        const long long n = (a.walk ? P : 0) + (long long)L;
        if (rows <= kRowsMax) {
            a.by_own = AttnBy::rows;
            cut_rows(n, groups, &a.parts_own, &a.chunk_own);
        } else {
            a.by_own = AttnBy::tiles;
            cut_tiles((a.walk ? tiles(P, 128) : 0) + tiles(L, 128), tiles(rows, 256) * groups, &a.parts_own, &a.chunk_own);
        }
    }
    const int parts = a.parts_own + a.parts_shared;
    if (parts == 1) return 0;
    return (size_t)parts * a.B * a.T * a.Hq * (a.d + 1) * 4;
}

template <int DIM, typename T>
static void launch_simple(const AttnArgs& a, cudaStream_t s) {
    const dim3 grid((a.T * a.Gq + kAtRows - 1) / kAtRows, a.Hkv, a.B);
    attn_kernel<DIM, T><<<grid, 256, 0, s>>>(a);
}

cudaError_t launch_attn(const AttnArgs& a, int num_sms, int* launches, cudaStream_t s) {
    *launches = 0;
    if (a.by_own == AttnBy::simple) {
        a.d == 128 ? launch_simple<128, float>(a, s) : launch_simple<64, float>(a, s);
        ++*launches;
        return cudaGetLastError();
    }
    cudaError_t e = cudaSuccess;
    auto run = [&](cudaError_t x) {
        e = x;
        ++*launches;
        return x == cudaSuccess;
    };
    if (a.by_shared == AttnBy::tiles && !run(launch_attn_tc(a, 1, num_sms, s))) return e;
    if (a.by_own == AttnBy::tiles && !run(launch_attn_tc(a, 0, num_sms, s))) return e;
    if ((a.by_shared == AttnBy::rows || a.by_own == AttnBy::rows) && !run(launch_attn_rows(a, s))) return e;
    if (a.part_o) {
        const unsigned grid = (unsigned)(((size_t)a.B * a.T * a.Hq + 3) / 4);
        if (a.d == 128) attn_join_kernel<128, __nv_bfloat16><<<grid, 128, 0, s>>>(a);
        else attn_join_kernel<64, __nv_bfloat16><<<grid, 128, 0, s>>>(a);
        run(cudaGetLastError());
    }
    return e;
}

}  // namespace lola
