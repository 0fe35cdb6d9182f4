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

cudaError_t launch_attn(const AttnArgs& a, cudaStream_t s) {
    const dim3 grid((a.T * a.Gq + kAtRows - 1) / kAtRows, a.Hkv, a.B);
    const bool bf = a.dtype == 1;
    if (a.d == 128) {
        if (bf) attn_kernel<128, __nv_bfloat16><<<grid, 256, 0, s>>>(a);
        else attn_kernel<128, float><<<grid, 256, 0, s>>>(a);
    } else {
        if (bf) attn_kernel<64, __nv_bfloat16><<<grid, 256, 0, s>>>(a);
        else attn_kernel<64, float><<<grid, 256, 0, s>>>(a);
    }
    return cudaGetLastError();
}

}  // namespace lola
