// Attention of several query tokens per request over the packed cache and over the drafted
// tokens themselves (sm_100a): the plain form, one warp per query row.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kvq_device.cuh"
#include "kvq_internal.h"
#include "kvq_quant.cuh"

namespace kvq {
namespace {

constexpr float kLog2eT = 1.4426950408889634f;

__device__ __forceinline__ float field_value(const uint8_t *codes, const uint8_t *sz, int role, bool per_token, int u,
                                             int d, int D, int bits) {
    int word, bit;
    quant::code_place(role, u & 15, d, D, bits, word, bit);
    const uint32_t w = reinterpret_cast<const uint32_t *>(codes + (u >> 4) * 2 * D * bits)[word];
    const int nj = D / 32;
    const int so = per_token ? quant::tok_sz_off(u, d / 32, nj) : quant::chan_sz_off(d);
    const int zo = so + (per_token ? 4 * nj : 4);
    return fmaf(static_cast<float>((w >> bit) & ((1u << bits) - 1u)),
                __half2float(*reinterpret_cast<const __half *>(sz + so)),
                __half2float(*reinterpret_cast<const __half *>(sz + zo)));
}

__global__ void __launch_bounds__(128) tree_row_kernel(const TreeParams p, int D, int bk, int bv, int kmode) {
    pdl_enter();
    __shared__ float qs[4][128], ps[4][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int Hq = p.Hkv * p.G;
    const long long row = static_cast<long long>(blockIdx.x) * 4 + warp;   // (b T + t) Hq + hq
    if (row >= static_cast<long long>(p.B) * p.T * Hq) return;
    const int hq = static_cast<int>(row % Hq), t = static_cast<int>(row / Hq % p.T), b = static_cast<int>(row / Hq / p.T);
    const int nq = p.len.queries(b), L = p.len.len(b), h = hq / p.G;
    if (t >= nq) return;
    const long long unit = static_cast<long long>(b) * p.Hkv + h;
    const int rec_bytes = 4 * D * bk + 4 * D + 4 * D * bv + 4 * D;
    const int depth = p.depth ? p.depth[b * p.T + t] : t;
    const int pos = L + p.pos0 + (p.kd ? depth : 0);
    const float slope = p.alibi ? p.alibi[hq] : 0.f;
    for (int d = lane; d < D; d += 32) qs[warp][d] = quant::bf16_to_f32(p.q[row * D + d]);
    __syncwarp();
    float m = -INFINITY, l = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
    const int nk = p.kd ? nq : 0;
    for (int t0 = 0; t0 < L + nk;) {
        const bool cached = t0 < L;
        const int n = cached ? min(32, L - t0) : min(32, L + nk - t0);
        const int blk = t0 >> 5, j0 = t0 - L;
        const uint8_t *rec = cached ? p.rec + rec_index(p.btab, b, p.Hkv, h, p.cap_blk, blk) * rec_bytes : nullptr;
        const bool open = cached && kmode == 0 && blk == (L >> 5);
        float s = -INFINITY;
        if (lane < n) {
            bool see = true;
            int kpos = t0 + lane;
            const uint16_t *krow = nullptr;
            if (!cached) {
                const int j = j0 + lane;
                see = p.mask ? (p.mask[(static_cast<long long>(b) * p.T + t) * p.mask_words + (j >> 5)] >> (j & 31)) & 1
                             : j <= t;
                kpos = L + (p.depth ? p.depth[b * p.T + j] : j);
                krow = p.kd + (unit * p.T + j) * D;
            } else if (open) krow = p.res + (unit * 32 + lane) * D;
            if (p.window && pos - kpos >= p.window) see = false;
            if (see) {
                float a = 0.f;
                for (int d = 0; d < D; ++d)
                    a = fmaf(qs[warp][d],
                             krow ? quant::bf16_to_f32(krow[d])
                                  : field_value(rec, rec + 4 * D * bk, 0, kmode == 1, lane, d, D, bk), a);
                a *= p.scale;
                if (p.cap > 0.f) a = p.cap * tanhf(a / p.cap);
                s = a - slope * static_cast<float>(pos - kpos);
            }
        }
        float mx = s;
        for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        const float mn = fmaxf(m, mx);
        if (mn > -INFINITY || __any_sync(0xffffffffu, s != s)) {
            const float al = exp2f((m - mn) * kLog2eT);
            const float e = s == -INFINITY ? 0.f : exp2f((s - mn) * kLog2eT);
            ps[warp][lane] = e;
            float sum = e;
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            const float a0 = m == -INFINITY ? 0.f : al;
            l = l * a0 + sum;
            m = mn;
            __syncwarp();
            for (int c = 0; c < D / 32; ++c) {
                const int d = 32 * c + lane;
                float a = acc[c] * a0;
                for (int u = 0; u < n; ++u) {
                    const float w = ps[warp][u];
                    if (w == 0.f) continue;
                    const float v = cached ? field_value(rec + 4 * D * bk + 4 * D, rec + 4 * D * bk + 4 * D + 4 * D * bv, 1,
                                                         true, u, d, D, bv)
                                           : quant::bf16_to_f32(p.vd[(unit * p.T + j0 + u) * D + d]);
                    a = fmaf(w, v, a);
                }
                acc[c] = a;
            }
            __syncwarp();
        }
        t0 += n;
    }
    for (int c = 0; c < D / 32; ++c) {
        const float o = l == 0.f ? 0.f : acc[c] / l;
        if (p.out_fp32) reinterpret_cast<float *>(p.out)[row * D + 32 * c + lane] = o;
        else reinterpret_cast<__nv_bfloat16 *>(p.out)[row * D + 32 * c + lane] = __float2bfloat16_rn(o);
    }
}

}  // namespace

int tree_row_groups(int rows) { return (rows + 255) / 256; }
int tree_max_splits(int, int, int) { return 1; }

cudaError_t launch_tree(const TreeParams &p, int D, int bk, int bv, int kmode, cudaStream_t st) {
    const long long rows = static_cast<long long>(p.B) * p.T * p.Hkv * p.G;
    cudaError_t e = launch_pdl(tree_row_kernel, dim3(static_cast<unsigned>((rows + 3) / 4)), dim3(128), 0, st, p, D, bk, bv,
                               kmode);
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_tree_merge(const TreeParams &, int, cudaStream_t) { return cudaSuccess; }

}  // namespace kvq
