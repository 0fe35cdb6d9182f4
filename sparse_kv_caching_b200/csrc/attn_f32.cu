// Exact attention, f32 inputs: f32 multiply-adds throughout (the tensor cores
// round f32 operands to 10 bits of mantissa), the same online softmax as the bf16
// kernels, keys walked as one sequence: the shared ones (where the rows read
// them), then the sequence's own, a range of them per CTA.
//
// attn_f32_rows_kernel, few rows: bound by HBM (8 d bytes a key).  Four rows per
// CTA; eight lanes share a key, so K and V rows go from global memory to registers
// in 128-byte pieces with no staging, each lane keeping its d / 8 elements of the
// four queries and of O.  A score takes three shuffles for four rows and keys at
// once; each eighth of a warp has a softmax state of its own until the end.
//
// attn_f32_tile_kernel, many rows: bound by the multiply-adds (2 d per row and key
// for each product).  64 rows x 64 keys (d = 128: 32) per step, 4 rows x 4 keys (2) of the scores and
// 4 rows x d / 16 columns of O per thread, operands from shared memory in 16-byte
// words (K rows padded by one: no bank conflicts); the next step's keys land meanwhile.
// B200: 2 x 333 queries x 1001 states, 12/4 heads, d 64: 68 us, 23 TFLOP/s with the join; the
// rows kernel, 7 tokens after 4095 shared keys, 6/2 heads, d 64: 12 us.
#include "attn.h"
#include "device_common.cuh"
#include "umma.cuh"

namespace lola {

constexpr int kFrRows = 4, kFrThreads = 128, kFrUnroll = 2;
constexpr int kFtRows = 64, kFtThreads = 256;

// What a CTA reads: the group's rows and a range [lo, hi) of the walk, whose first np0 keys are shared.
struct F32Work {
    int g, n0, R, np0, lo, hi, len, part;
    const float *ksh, *vsh, *kow, *vow;
};
__device__ __forceinline__ F32Work f32_work(const AttnArgs& a, int i, int packed) {
    F32Work w;
    const int parts = packed ? a.parts_shared : a.parts_own, chunk = packed ? a.chunk_shared : a.chunk_own;
    w.part = i % parts;
    i /= parts;
    w.g = i % a.Hkv;
    const int b = i / a.Hkv;
    w.n0 = b * a.T;
    w.R = (packed ? a.B : 1) * a.T * a.Gq;
    w.np0 = packed || a.walk ? a.shared.n : 0;
    w.len = packed ? 0 : own_length(a, b);
    w.lo = w.part * chunk;
    w.hi = (int)min((long long)w.np0 + w.len, (long long)w.lo + chunk);
    w.part += packed ? 0 : a.parts_shared;
    w.ksh = (const float*)a.shared.k + (long long)w.g * a.shared.kh;
    w.vsh = (const float*)a.shared.v + (long long)w.g * a.shared.vh;
    w.kow = (const float*)a.own.k + b * a.own.kb + (long long)w.g * a.own.kh;
    w.vow = (const float*)a.own.v + b * a.own.vb + (long long)w.g * a.own.vh;
    return w;
}
__device__ __forceinline__ const float* f32_key(const AttnArgs& a, const F32Work& w, int key) {
    return key < w.np0 ? w.ksh + (long long)key * a.shared.ks : w.kow + (long long)(key - w.np0) * a.own.ks;
}
__device__ __forceinline__ const float* f32_value(const AttnArgs& a, const F32Work& w, int key) {
    return key < w.np0 ? w.vsh + (long long)key * a.shared.vs : w.vow + (long long)(key - w.np0) * a.own.vs;
}

// One row's result, to y and lse or as a part; `o` holds 4 of its columns from column c.
__device__ __forceinline__ void f32_store(const AttnArgs& a, const F32Work& w, size_t at, int c, float4 o, float m, float l) {
    const float inv = l == 0.f ? 0.f : 1.f / l, l2 = l == 0.f ? -INFINITY : m + log2f(l);
    o.x *= inv; o.y *= inv; o.z *= inv; o.w *= inv;
    if (a.part_o) {
        const size_t p = (size_t)w.part * a.B * a.T * a.Hq + at;
        *reinterpret_cast<float4*>(a.part_o + p * a.d + c) = o;
        if (c == 0) a.part_l[p] = l2;
    } else {
        *reinterpret_cast<float4*>((float*)a.y + at * a.d + c) = o;
        if (a.lse && c == 0) a.lse[at] = l2 * 0.6931471805599453f;
    }
}

__device__ __forceinline__ float dot4(float4 x, float4 y, float s) {
    return fmaf(x.x, y.x, fmaf(x.y, y.y, fmaf(x.z, y.z, fmaf(x.w, y.w, s))));
}

template <int DIM>
__global__ void __launch_bounds__(kFrThreads) attn_f32_rows_kernel(const __grid_constant__ AttnArgs a) {
    constexpr int NF = DIM / 32;                  // 16-byte words of a row per lane (of 8)
    constexpr int STEP = kFrUnroll * 4 * (kFrThreads / 32);
    __shared__ float so[kFrThreads / 32][kFrRows][DIM];
    __shared__ float2 sml[kFrThreads / 32][kFrRows];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, c8 = lane & 7, grp = lane >> 3;
    attn_let_next_begin();
    const F32Work w = f32_work(a, blockIdx.x, 0);
    const int r0 = blockIdx.y * kFrRows;
    float4 q[kFrRows][NF], o[kFrRows][NF];
    float m[kFrRows], l[kFrRows];
    int lim[kFrRows];
#pragma unroll
    for (int i = 0; i < kFrRows; ++i) {
        const bool ok = r0 + i < w.R;
        const RowAt x = row_at(a, w.n0, w.g, ok ? r0 + i : 0);
        lim[i] = ok ? min(w.hi, w.np0 + own_visible(a, w.len, x.t)) : 0;
        m[i] = -INFINITY;
        l[i] = 0.f;
#pragma unroll
        for (int u = 0; u < NF; ++u) {
            q[i][u] = *reinterpret_cast<const float4*>((const float*)a.q + x.q + 4 * (c8 + 8 * u));
            o[i][u] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
    }
    for (int k0 = w.lo + warp * 4 * kFrUnroll + grp; k0 - grp < w.hi; k0 += STEP) {
        float4 kk[kFrUnroll][NF], vv[kFrUnroll][NF];
#pragma unroll
        for (int u = 0; u < kFrUnroll; ++u) {
            const int key = k0 + 4 * u;
            const bool ok = key < w.hi;
            const float4* kp = reinterpret_cast<const float4*>(ok ? f32_key(a, w, key) : nullptr) + c8;
            const float4* vp = reinterpret_cast<const float4*>(ok ? f32_value(a, w, key) : nullptr) + c8;
#pragma unroll
            for (int i = 0; i < NF; ++i) {
                kk[u][i] = ok ? kp[8 * i] : make_float4(0.f, 0.f, 0.f, 0.f);
                vv[u][i] = ok ? vp[8 * i] : make_float4(0.f, 0.f, 0.f, 0.f);
            }
        }
#pragma unroll
        for (int i = 0; i < kFrRows; ++i) {
            float x[kFrUnroll], mn = m[i];
#pragma unroll
            for (int u = 0; u < kFrUnroll; ++u) {
                float s = 0.f;
#pragma unroll
                for (int j = 0; j < NF; ++j) s = dot4(q[i][j], kk[u][j], s);
                s += __shfl_xor_sync(0xffffffffu, s, 1);
                s += __shfl_xor_sync(0xffffffffu, s, 2);
                s += __shfl_xor_sync(0xffffffffu, s, 4);
                x[u] = k0 + 4 * u < lim[i] ? s * a.scale_log2 : -INFINITY;
                mn = fmaxf(mn, x[u]);
            }
            const float ref = mn == -INFINITY ? 0.f : mn, f = exp2f(m[i] - ref);
            m[i] = mn;
            l[i] *= f;
#pragma unroll
            for (int j = 0; j < NF; ++j) { o[i][j].x *= f; o[i][j].y *= f; o[i][j].z *= f; o[i][j].w *= f; }
#pragma unroll
            for (int u = 0; u < kFrUnroll; ++u) {
                const float p = exp2f(x[u] - ref);
                l[i] += p;
#pragma unroll
                for (int j = 0; j < NF; ++j) {
                    o[i][j].x = fmaf(p, vv[u][j].x, o[i][j].x); o[i][j].y = fmaf(p, vv[u][j].y, o[i][j].y);
                    o[i][j].z = fmaf(p, vv[u][j].z, o[i][j].z); o[i][j].w = fmaf(p, vv[u][j].w, o[i][j].w);
                }
            }
        }
    }
    // the four eighth-warp states of each warp, then the warps'
#pragma unroll
    for (int i = 0; i < kFrRows; ++i) {
        float mx = fmaxf(m[i], __shfl_xor_sync(0xffffffffu, m[i], 8));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
        const float f = exp2f(m[i] - (mx == -INFINITY ? 0.f : mx));
        float s = l[i] * f;
        s += __shfl_xor_sync(0xffffffffu, s, 8);
        s += __shfl_xor_sync(0xffffffffu, s, 16);
        if (lane == 0) sml[warp][i] = make_float2(mx, s);
#pragma unroll
        for (int j = 0; j < NF; ++j) {
            float4 z = o[i][j];
            z.x *= f; z.y *= f; z.z *= f; z.w *= f;
#pragma unroll
            for (int k = 8; k <= 16; k += 8) {
                z.x += __shfl_xor_sync(0xffffffffu, z.x, k); z.y += __shfl_xor_sync(0xffffffffu, z.y, k);
                z.z += __shfl_xor_sync(0xffffffffu, z.z, k); z.w += __shfl_xor_sync(0xffffffffu, z.w, k);
            }
            if (grp == 0) *reinterpret_cast<float4*>(&so[warp][i][4 * (c8 + 8 * j)]) = z;
        }
    }
    __syncthreads();
    for (int i = tid; i < kFrRows * (DIM / 4); i += kFrThreads) {
        const int r = i / (DIM / 4), c = i % (DIM / 4) * 4;
        if (r0 + r >= w.R) break;
        float mx = -INFINITY, sum = 0.f;
#pragma unroll
        for (int k = 0; k < kFrThreads / 32; ++k) mx = fmaxf(mx, sml[k][r].x);
        const float ref = mx == -INFINITY ? 0.f : mx;
        float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < kFrThreads / 32; ++k) {
            const float f = exp2f(sml[k][r].x - ref);
            const float4 x = *reinterpret_cast<const float4*>(&so[k][r][c]);
            sum = fmaf(sml[k][r].y, f, sum);
            z.x = fmaf(x.x, f, z.x); z.y = fmaf(x.y, f, z.y); z.z = fmaf(x.z, f, z.z); z.w = fmaf(x.w, f, z.w);
        }
        f32_store(a, w, row_at(a, w.n0, w.g, r0 + r).o, c, z, ref, sum);
    }
}

template <int DIM>
struct F32Tile {
    static constexpr int KEYS = DIM == 64 ? 64 : 32, KPT = KEYS / 16;   // keys of a step (two CTAs share an SM), of a thread
    static constexpr int LQ = DIM + 4, LP = KEYS + 4;
    static constexpr int KV = KEYS * LQ + KEYS * DIM;                   // a stage: K (padded rows), then V
    static constexpr int Q = 0, ST = Q + kFtRows * LQ, PP = ST + 2 * KV, WORDS = PP + kFtRows * LP;
};

template <int DIM>
__global__ void __launch_bounds__(kFtThreads, 2) attn_f32_tile_kernel(const __grid_constant__ AttnArgs a, int packed) {
    using Sh = F32Tile<DIM>;
    constexpr int NC = DIM / 64, LQ = Sh::LQ, LP = Sh::LP, KEYS = Sh::KEYS, KPT = Sh::KPT;
    extern __shared__ __align__(16) float fs[];
    float *sq = fs + Sh::Q, *sp = fs + Sh::PP;
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const int row_tiles = ((packed ? a.B : 1) * a.T * a.Gq + kFtRows - 1) / kFtRows;
    attn_let_next_begin();
    const F32Work w = f32_work(a, blockIdx.x / row_tiles, packed);     // neighbours read the same keys
    const int r0 = (blockIdx.x % row_tiles) * kFtRows;
    for (int i = tid; i < kFtRows * DIM / 4; i += kFtThreads) {
        const int r = i / (DIM / 4), c = i % (DIM / 4) * 4;
        const bool ok = r0 + r < w.R;
        umma::cp_async16_zfill(sq + r * LQ + c, (const float*)a.q + row_at(a, w.n0, w.g, ok ? r0 + r : 0).q + c, ok);
    }
    float m[4], l[4];
    ulonglong2 o[4][NC];                          // four columns each, in pairs
    int lim[4], most = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = r0 + 4 * ty + i;
        lim[i] = r < w.R ? min(w.hi, w.np0 + own_visible(a, w.len, row_at(a, w.n0, w.g, r).t)) : 0;
        m[i] = -INFINITY;
        l[i] = 0.f;
#pragma unroll
        for (int j = 0; j < NC; ++j) o[i][j] = make_ulonglong2(0ull, 0ull);
    }
    {   // the last row of the tile reads furthest
        const int r = min(w.R, r0 + kFtRows) - 1;
        most = packed ? w.hi : min(w.hi, w.np0 + own_visible(a, w.len, row_at(a, w.n0, w.g, r).t));
    }
    // the keys of a step while the one before is computed
    auto fetch = [&](int k0, int stage) {
        if (k0 < most) {
            float *sk = fs + Sh::ST + stage * Sh::KV, *sv = sk + KEYS * LQ;
            for (int i = tid; i < KEYS * DIM / 4; i += kFtThreads) {
                const int r = i / (DIM / 4), c = i % (DIM / 4) * 4, key = k0 + r;
                const bool ok = key < w.hi;
                umma::cp_async16_zfill(sk + r * LQ + c, ok ? (const void*)(f32_key(a, w, key) + c) : a.q, ok);
                umma::cp_async16_zfill(sv + r * DIM + c, ok ? (const void*)(f32_value(a, w, key) + c) : a.q, ok);
            }
        }
        umma::cp_async_commit();
    };
    fetch(w.lo, 0);
    int stage = 0;
    for (int k0 = w.lo; k0 < most; k0 += KEYS, stage ^= 1) {
        fetch(most - k0 > KEYS ? k0 + KEYS : most, stage ^ 1);
        umma::cp_async_wait<1>();
        __syncthreads();
        const float *sk = fs + Sh::ST + stage * Sh::KV, *sv = sk + KEYS * LQ;
        // (pairs of multiply-adds: even dims in the low halves, odd ones in the high)
        unsigned long long s2[4][KPT];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int k = 0; k < KPT; ++k) s2[i][k] = 0ull;
#pragma unroll 4
        for (int c = 0; c < DIM; c += 4) {
            ulonglong2 kk[KPT];
#pragma unroll
            for (int k = 0; k < KPT; ++k) kk[k] = *reinterpret_cast<const ulonglong2*>(sk + (tx + 16 * k) * LQ + c);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const ulonglong2 x = *reinterpret_cast<const ulonglong2*>(sq + (4 * ty + i) * LQ + c);
#pragma unroll
                for (int k = 0; k < KPT; ++k) s2[i][k] = f2fma(x.y, kk[k].y, f2fma(x.x, kk[k].x, s2[i][k]));
            }
        }
        float s[4][KPT];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int k = 0; k < KPT; ++k) {
                float lo, hi;
                f2unpack(s2[i][k], lo, hi);
                s[i][k] = lo + hi;
            }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float mx = -INFINITY;
#pragma unroll
            for (int k = 0; k < KPT; ++k) {
                s[i][k] = k0 + tx + 16 * k < lim[i] ? s[i][k] * a.scale_log2 : -INFINITY;
                mx = fmaxf(mx, s[i][k]);
            }
#pragma unroll
            for (int k = 1; k < 16; k <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, k));
            const float mn = fmaxf(m[i], mx), ref = mn == -INFINITY ? 0.f : mn, f = exp2f(m[i] - ref);
            m[i] = mn;
            l[i] *= f;                            // this thread's keys only: summed at the end
#pragma unroll
            for (int k = 0; k < KPT; ++k) {
                const float p = exp2f(s[i][k] - ref);
                l[i] += p;
                sp[(4 * ty + i) * LP + tx + 16 * k] = p;
            }
#pragma unroll
            for (int j = 0; j < NC; ++j) {
                o[i][j].x = f2fma(o[i][j].x, f2pack(f, f), 0ull);
                o[i][j].y = f2fma(o[i][j].y, f2pack(f, f), 0ull);
            }
        }
        __syncwarp();                             // a row's weights are written and read by one warp
#pragma unroll 2
        for (int k = 0; k < KEYS; k += 4) {
            float4 p[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) p[i] = *reinterpret_cast<const float4*>(sp + (4 * ty + i) * LP + k);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
#pragma unroll
                for (int j = 0; j < NC; ++j) {
                    const ulonglong2 x = *reinterpret_cast<const ulonglong2*>(sv + (k + kk) * DIM + 64 * j + 4 * tx);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float y = kk == 0 ? p[i].x : kk == 1 ? p[i].y : kk == 2 ? p[i].z : p[i].w;
                        o[i][j].x = f2fma(f2pack(y, y), x.x, o[i][j].x);
                        o[i][j].y = f2fma(f2pack(y, y), x.y, o[i][j].y);
                    }
                }
        }
        __syncthreads();                          // the stage is free
    }
    umma::cp_async_wait<0>();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int k = 1; k < 16; k <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], k);
        const int r = r0 + 4 * ty + i;
        if (r >= w.R) continue;
        const size_t at = row_at(a, w.n0, w.g, r).o;
#pragma unroll
        for (int j = 0; j < NC; ++j) {
            float4 y;
            f2unpack(o[i][j].x, y.x, y.y);
            f2unpack(o[i][j].y, y.z, y.w);
            f32_store(a, w, at, 64 * j + 4 * tx, y, m[i], l[i]);
        }
    }
}

cudaError_t launch_attn_f32_rows(const AttnArgs& a, cudaStream_t s) {
    const dim3 grid(a.parts_own * a.Hkv * a.B, (a.T * a.Gq + kFrRows - 1) / kFrRows);
    if (a.d == 128) attn_f32_rows_kernel<128><<<grid, kFrThreads, 0, s>>>(a);
    else attn_f32_rows_kernel<64><<<grid, kFrThreads, 0, s>>>(a);
    return cudaGetLastError();
}

template <int DIM>
static cudaError_t launch_tile_t(const AttnArgs& a, int packed, cudaStream_t s) {
    constexpr int bytes = F32Tile<DIM>::WORDS * 4;
    static std::atomic<unsigned long long> done{0};
    cudaError_t e = allow_smem(attn_f32_tile_kernel<DIM>, bytes, &done);
    if (e != cudaSuccess) return e;
    const int rows = (packed ? a.B : 1) * a.T * a.Gq;
    const unsigned grid = (rows + kFtRows - 1) / kFtRows * (packed ? a.parts_shared * a.Hkv : a.parts_own * a.Hkv * a.B);
    attn_f32_tile_kernel<DIM><<<grid, kFtThreads, bytes, s>>>(a, packed);
    return cudaGetLastError();
}

cudaError_t launch_attn_f32_tiles(const AttnArgs& a, int packed, cudaStream_t s) {
    return a.d == 128 ? launch_tile_t<128>(a, packed, s) : launch_tile_t<64>(a, packed, s);
}

}  // namespace lola
