// Exact attention for few rows per kv head (decode steps, short drafts), bf16.
//
// A group's R <= 32 rows (queries x heads of the kv group) read N keys: 4 R d N
// operations on 4 d N bytes, R operations a byte, so the kernel is bound by HBM
// as long as each key is read once for all its rows and enough loads are in
// flight.  One warp owns 16-key blocks (every kRwWarps-th of its CTA's range): it
// copies a block's K and V rows into its own ring of stages with cp.async two
// blocks ahead and never waits for another warp; S = Q K^T and O += P V run on
// the warp-level tensor instructions (m16n8k16: 16-row tiles of Q in registers,
// which a tile of 128 rows on the SM-level unit would leave almost empty).
// Softmax: running maximum and sum per row and warp, f32; the accumulator is
// rescaled only when a maximum rises.  P is fed as two bf16 parts (its rounding
// and the remainder): the second product is free under the loads and keeps the
// weights to 2^-16.  At the end the warps' (m, l, O) meet in shared memory.
// Rows of V that no query of the group may read are filled with zeros.
#include "attn.h"
#include "umma.cuh"

namespace lola {

constexpr int kRwWarps = 4, kRwKeys = 16, kRwStages = 3;

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

template <int DIM, int MT>
struct RowsShape {
    static constexpr int STAGE = 2 * kRwKeys * DIM * 2;               // K rows, then V rows
    static constexpr int WARP = kRwStages * STAGE;
    static constexpr int RED = MT * 16 * DIM * 4;                     // one warp's O, at the end
    static constexpr int BYTES = kRwWarps * WARP + kRwWarps * MT * 16 * 8;
    static_assert(RED <= WARP, "the stages hold a warp's O");
};

template <int DIM, int MT>
__global__ void __launch_bounds__(kRwWarps * 32) attn_rows_kernel(const __grid_constant__ AttnArgs a) {
    using Sh = RowsShape<DIM, MT>;
    using bf16 = __nv_bfloat16;
    constexpr int KC = DIM / 8;                 // 16-byte chunks of a key row
    constexpr int RB = DIM * 2;                 // its bytes
    extern __shared__ __align__(128) uint8_t smem[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

    // ---- which rows, which keys ----
    const int n_sh = a.by_shared == AttnBy::rows ? a.parts_shared * a.Hkv : 0;      // CTAs of the shared group
    int g, b = 0, part, lo, hi, n0, R, np0;     // np0: keys of the walk that are shared ones
    if ((int)blockIdx.x < n_sh) {
        part = blockIdx.x % a.parts_shared;
        g = blockIdx.x / a.parts_shared;
        n0 = 0;
        R = a.B * a.T * a.Gq;
        np0 = a.shared.n;
        lo = part * a.chunk_shared;
        hi = (int)min((long long)np0, (long long)lo + a.chunk_shared);
    } else {
        int i = blockIdx.x - n_sh;
        part = i % a.parts_own;
        i /= a.parts_own;
        g = i % a.Hkv;
        b = i / a.Hkv;
        n0 = b * a.T;
        R = a.T * a.Gq;
        np0 = a.walk ? a.shared.n : 0;
        lo = part * a.chunk_own;
        hi = (int)min((long long)np0 + own_length(a, b), (long long)lo + a.chunk_own);
        part += a.parts_shared;
    }
    const int len = (int)blockIdx.x < n_sh ? 0 : own_length(a, b);
    const bf16* ksh = (const bf16*)a.shared.k + (long long)g * a.shared.kh;
    const bf16* vsh = (const bf16*)a.shared.v + (long long)g * a.shared.vh;
    const bf16* kow = (const bf16*)a.own.k + b * a.own.kb + (long long)g * a.own.kh;
    const bf16* vow = (const bf16*)a.own.v + b * a.own.vb + (long long)g * a.own.vh;

    uint8_t* ring = smem + warp * Sh::WARP;
    const int nblk = max(0, (hi - lo + kRwKeys - 1) / kRwKeys);
    const int mine = nblk > warp ? (nblk - warp + kRwWarps - 1) / kRwWarps : 0;
    // copy block j of this warp into its stage: lanes take one 16-byte chunk of a row each
    auto fetch = [&](int j) {
        uint8_t* st = ring + (j % kRwStages) * Sh::STAGE;
        const int k0 = lo + (warp + j * kRwWarps) * kRwKeys;
        constexpr int RPI = 32 / KC;            // rows per pass
#pragma unroll
        for (int it = 0; it < kRwKeys / RPI; ++it) {
            const int r = it * RPI + lane / KC, c = lane % KC, key = k0 + r;
            const bool ok = key < hi, sh = key < np0;
            const long long i = ok ? (sh ? key : key - np0) : 0;
            const bf16* kp = (sh ? ksh + i * a.shared.ks : kow + i * a.own.ks) + 8 * c;
            const bf16* vp = (sh ? vsh + i * a.shared.vs : vow + i * a.own.vs) + 8 * c;
            const uint32_t off = r * RB + ((c ^ (r & 7)) << 4);
            umma::cp_async16_zfill(st + off, ok ? (const void*)kp : a.q, ok);
            umma::cp_async16_zfill(st + kRwKeys * RB + off, ok ? (const void*)vp : a.q, ok);
        }
    };
#pragma unroll
    for (int j = 0; j < kRwStages - 1; ++j) {
        if (j < mine) fetch(j);
        umma::cp_async_commit();
    }

    // ---- queries: A fragments of 16-row tiles (row lane/4 and + 8, dims 2 (lane%4) and + 8) ----
    uint32_t qf[MT][DIM / 16][4];
    int lim[MT][2];                             // keys of the walk that each of this lane's rows reads
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
            const int r = mt * 16 + hh * 8 + lane / 4;
            const bool ok = r < R;
            const RowAt x = row_at(a, n0, g, ok ? r : 0);
            const uint32_t* qp = reinterpret_cast<const uint32_t*>((const bf16*)a.q + x.q) + lane % 4;
            lim[mt][hh] = np0 + own_visible(a, len, x.t);
#pragma unroll
            for (int kk = 0; kk < DIM / 16; ++kk) {
                qf[mt][kk][hh] = ok ? qp[8 * kk] : 0u;
                qf[mt][kk][hh + 2] = ok ? qp[8 * kk + 4] : 0u;
            }
        }

    float o[MT][DIM / 8][4], m[MT][2], l[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
        for (int n = 0; n < DIM / 8; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[mt][n][i] = 0.f;
        m[mt][0] = m[mt][1] = -INFINITY;
        l[mt][0] = l[mt][1] = 0.f;
    }
    const uint32_t ring_s = umma::smem_addr(ring);
    // ldmatrix addresses: lane i gives row (i % 8) of 8 x 8 matrix i / 8
    const int krow = (lane & 7) + ((lane >> 4) << 3), kch = (lane >> 3) & 1;      // K: matrices (keys, dims) 00 01 10 11
    const int vrow = (lane & 7) + (((lane >> 3) & 1) << 3), vch = lane >> 4;      // V: (keys, dims) 00 10 01 11
    for (int j = 0; j < mine; ++j) {
        umma::cp_async_wait<kRwStages - 2>();
        __syncwarp();
        if (j + kRwStages - 1 < mine) fetch(j + kRwStages - 1);       // into the stage read at j - 1
        umma::cp_async_commit();
        const uint32_t ks = ring_s + (j % kRwStages) * Sh::STAGE, vs = ks + kRwKeys * RB;
        const int k0 = lo + (warp + j * kRwWarps) * kRwKeys;
        float s[MT][2][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[mt][0][i] = s[mt][1][i] = 0.f;
#pragma unroll
        for (int kk = 0; kk < DIM / 16; ++kk) {
            uint32_t kf[4];
            rw_ldsm(kf, ks + krow * RB + (((2 * kk + kch) ^ (krow & 7)) << 4));
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                rw_mma(s[mt][0], qf[mt][kk], kf[0], kf[1]);
                rw_mma(s[mt][1], qf[mt][kk], kf[2], kf[3]);
            }
        }
        uint32_t ph[MT][4], pl[MT][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            float f[2];
            bool up = false;
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
                // this lane's keys: 2 (lane % 4) + {0, 1} of each 8-key tile
                float x[4], mx = -INFINITY;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int key = k0 + (i >> 1) * 8 + 2 * (lane & 3) + (i & 1);
                    x[i] = key < min(lim[mt][hh], hi) ? s[mt][i >> 1][2 * hh + (i & 1)] * a.scale_log2 : -INFINITY;
                    mx = fmaxf(mx, x[i]);
                }
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                const float mn = fmaxf(m[mt][hh], mx), ref = mn == -INFINITY ? 0.f : mn;
                f[hh] = rw_ex2(m[mt][hh] - ref);
                up |= mn != m[mt][hh];
                m[mt][hh] = mn;
                float sum = 0.f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[i] = rw_ex2(x[i] - ref);
                    sum += x[i];
                }
                l[mt][hh] = l[mt][hh] * f[hh] + sum;                  // this lane's keys only: summed over lanes at the end
                rw_split(x[0], x[1], ph[mt][hh], pl[mt][hh]);         // A fragment: keys 2 (lane%4), then + 8
                rw_split(x[2], x[3], ph[mt][hh + 2], pl[mt][hh + 2]);
            }
            if (__any_sync(0xffffffffu, up)) {
#pragma unroll
                for (int n = 0; n < DIM / 8; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[mt][n][i] *= f[i >> 1];
            }
        }
#pragma unroll
        for (int n2 = 0; n2 < DIM / 16; ++n2) {
            uint32_t vf[4];
            rw_ldsm_t(vf, vs + vrow * RB + (((2 * n2 + vch) ^ (vrow & 7)) << 4));
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                rw_mma(o[mt][2 * n2], ph[mt], vf[0], vf[1]);
                rw_mma(o[mt][2 * n2 + 1], ph[mt], vf[2], vf[3]);
                rw_mma(o[mt][2 * n2], pl[mt], vf[0], vf[1]);
                rw_mma(o[mt][2 * n2 + 1], pl[mt], vf[2], vf[3]);
            }
        }
    }

    // ---- the warps' sums meet: O in the (free) stages, m and l behind them ----
    umma::cp_async_wait<0>();
    __syncwarp();
    float* red = reinterpret_cast<float*>(ring);
    float2* ml = reinterpret_cast<float2*>(smem + kRwWarps * Sh::WARP);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
            float x = l[mt][hh];
            x += __shfl_xor_sync(0xffffffffu, x, 1);
            x += __shfl_xor_sync(0xffffffffu, x, 2);
            const int r = mt * 16 + hh * 8 + lane / 4;
            if ((lane & 3) == 0) ml[warp * MT * 16 + r] = make_float2(m[mt][hh], x);
            if (r < R) {
#pragma unroll
                for (int n = 0; n < DIM / 8; ++n)
                    *reinterpret_cast<float2*>(red + r * DIM + 8 * n + 2 * (lane & 3)) =
                        make_float2(o[mt][n][2 * hh], o[mt][n][2 * hh + 1]);
            }
        }
    __syncthreads();
    const bool whole = a.part_o == nullptr;
    const size_t rows_all = (size_t)a.B * a.T * a.Hq;
    for (int i = tid; i < R * (DIM / 4); i += kRwWarps * 32) {
        const int r = i / (DIM / 4), c = i % (DIM / 4) * 4;
        float mx = -INFINITY;
#pragma unroll
        for (int w = 0; w < kRwWarps; ++w) mx = fmaxf(mx, ml[w * MT * 16 + r].x);
        const float ref = mx == -INFINITY ? 0.f : mx;
        float sum = 0.f;
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kRwWarps; ++w) {
            const float2 z = ml[w * MT * 16 + r];
            const float f = rw_ex2(z.x - ref);
            const float4 x = *reinterpret_cast<const float4*>(smem + w * Sh::WARP + (r * DIM + c) * 4);
            sum = fmaf(z.y, f, sum);
            y.x = fmaf(x.x, f, y.x); y.y = fmaf(x.y, f, y.y); y.z = fmaf(x.z, f, y.z); y.w = fmaf(x.w, f, y.w);
        }
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        y.x *= inv; y.y *= inv; y.z *= inv; y.w *= inv;
        const size_t at = row_at(a, n0, g, r).o;
        const float l2 = sum == 0.f ? -INFINITY : ref + log2f(sum);
        if (whole) {
            *reinterpret_cast<uint2*>((bf16*)a.y + at * DIM + c) = make_uint2(rw_pack(y.x, y.y), rw_pack(y.z, y.w));
            if (a.lse && c == 0) a.lse[at] = l2 * 0.6931471805599453f;
        } else {
            *reinterpret_cast<float4*>(a.part_o + (part * rows_all + at) * DIM + c) = y;
            if (c == 0) a.part_l[part * rows_all + at] = l2;
        }
    }
}

template <int DIM, int MT>
static cudaError_t launch_rows_t(const AttnArgs& a, cudaStream_t s) {
    using Sh = RowsShape<DIM, MT>;
    cudaError_t e = cudaFuncSetAttribute(attn_rows_kernel<DIM, MT>, cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::BYTES);
    if (e != cudaSuccess) return e;
    const unsigned grid = (a.by_shared == AttnBy::rows ? a.parts_shared * a.Hkv : 0) +
                          (a.by_own == AttnBy::rows ? a.parts_own * a.Hkv * a.B : 0);
    attn_rows_kernel<DIM, MT><<<grid, kRwWarps * 32, Sh::BYTES, s>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_attn_rows(const AttnArgs& a, cudaStream_t s) {
    const int rows = (a.by_shared == AttnBy::rows ? a.B : 1) * a.T * a.Gq;
    if (a.d == 128) return rows <= 16 ? launch_rows_t<128, 1>(a, s) : launch_rows_t<128, 2>(a, s);
    return rows <= 16 ? launch_rows_t<64, 1>(a, s) : launch_rows_t<64, 2>(a, s);
}

}  // namespace lola
