// RMS norm of query and key heads, rotation by position, and the split of a projection's
// rows into q (by token) and K, V (by kv head), one pass over the data (sm_100a).
//
//   y = x / sqrt(mean(x^2) + eps) * w                      (per head, if a weight is given)
//   (a, b) -> (a cos f - b sin f, b cos f + a sin f),  f = position * inv_freq[i]
//
// The work is a copy: every row is read once and written once (bound: HBM; for a decode
// step: the launch).  A row is held by D / 16 threads, two 16-byte chunks each, chosen so
// that a thread has both ends of its rotation pairs: chunks u and u + rot / 16 (which hold
// channels i and i + rot / 2; adjacent pairs sit inside one chunk) for the rotated part,
// the remaining chunks two by two.  The norm's sum is one shuffle tree over those threads.
// Angles: one (token, pair) per thread into shared memory, shared by the token's heads.  The
// angle in turns is reduced in fp64 (position * inv_freq reaches 2^30, fp32 would lose the
// fraction), its cosine and sine are taken in fp32 of the reduced value.  Sums and rotation
// are fp32; each output is rounded once to bf16.
#include <cuda_bf16.h>

#include "kvq_device.cuh"
#include "kvq_internal.h"

namespace kvq {
namespace {

constexpr int kRopeThreads = 384;   // the most threads of a CTA

__device__ __forceinline__ void bf16x8_to_f32(const uint4 &v, float *x) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ uint4 f32x8_to_bf16(const float *x) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&b);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// A CTA takes tpc tokens: as many as its threads hold, or more (4, 8 or 16: fewer barriers and angle
// steps per token, the next pass's rows fetched before this pass's are written) where the launch
// then still has six CTAs per SM, two rounds of the three that an SM holds.  Device time in us with
// 1 (as many as fit) / 4 / 8 / 16 tokens per CTA, 48 rows of 128 channels (Llama heads):
//   tokens   2,048: 16.4 / 16.9 / 22.0 / 21.3      8,192: 54.3 / 51.2 / 51.2 / 58.2
//            4,096: 29.2 / 27.1 / 30.7 / 39.9     12,000: 76.8 / 72.7 / 74.8 / 79.9
//           16,384: 101.4 / 94.2 / 93.2 / 93.2    65,536: 386 / 354 / 350 / 344 (72% of the copy rate)
// 36 rows (28 + 8 heads): 4,096 tokens 22.2 / 21.9 / 24.2 / 31.7, 16,384 tokens 77.9 / 76.8 / 73.7 /
// 73.8.  10 rows (4 tokens fit): 8,192 tokens 16.4 with 4, 16.8 with 8, the rule's worst of those
// measured.  Two tokens where one fits lose up to 26% (half-empty second passes).  A persistent
// grid that fetched across tokens: 140 us at 16,384 (78 registers: fewer threads in flight).  What
// bounds a long prompt: the L1 / shared-memory data path (80% of its wavefronts: a thread's angle pairs lie
// 64 bytes apart from its neighbour's) and issue (74%); DRAM is at 44%.  A decode step's 64 tokens (2.9 us)
// are bound by the launch.  Dynamic shared memory: tpc * rot / 2 (cos, sin) pairs.
template <int D>
__global__ void __launch_bounds__(kRopeThreads, 3) rope_kernel(const RopeParams p, int tpc) {
    pdl_enter();
    extern __shared__ float2 cs_s[];
    constexpr int TPR = D / 16;                    // threads per row
    const int rows = p.Hq + 2 * p.Hkv;             // rows of a token
    const int half = p.rot >> 1, rc = p.rot >> 4;  // pairs; threads with rotated chunks
    const unsigned tokens = static_cast<unsigned>(p.B) * p.n;   // below 2^31
    const int u = threadIdx.x % TPR;
    const int c0 = u < rc ? u : 2 * u, c1 = u < rc ? u + rc : 2 * u + 1;
    // blockDim is a multiple of 32 and TPR divides 32: a row's threads share a warp, and all
    // lanes of a warp run the same number of passes (inactive rows are clamped, not skipped)
    const int step = blockDim.x / TPR, first = threadIdx.x / TPR;
    auto tokens_of = [&](unsigned g) { return min(static_cast<unsigned>(tpc), tokens - g * tpc); };
    // row `it` of group g: its token (request b, index ti) and row
    auto place = [&](unsigned g, int it, unsigned &b, unsigned &ti, int &j, int &row) {
        const int last = static_cast<int>(tokens_of(g)) * rows - 1;
        it = min(it, last);
        j = tpc == 1 ? 0 : it / rows;
        row = it - j * rows;
        const unsigned tok = g * tpc + j;
        b = tok / p.n;
        ti = tok - b * p.n;
    };
    auto fetch = [&](unsigned g, int it, uint4 &v0, uint4 &v1) {
        unsigned b, ti;
        int j, row;
        place(g, it, b, ti, j, row);
        const uint16_t *s = p.qkv + b * p.batch_stride + ti * p.token_stride + static_cast<long long>(row) * D;
        v0 = *reinterpret_cast<const uint4 *>(s + 8 * c0);
        v1 = *reinterpret_cast<const uint4 *>(s + 8 * c1);
    };
    auto angles = [&](unsigned g, float2 *cs) {
        const int cnt = static_cast<int>(tokens_of(g)) * half;
        for (int k = threadIdx.x; k < cnt; k += blockDim.x) {
            const int j = k / half, i = k - j * half;
            const unsigned tok = g * tpc + j, b = tok / p.n, ti = tok - b * p.n;
            const double pos = static_cast<double>(p.len.len(b)) + (p.offset ? p.offset[tok] : static_cast<int>(ti));
            // turns = position * inv_freq / (2 pi): the fraction survives in fp64
            const double turns = pos * static_cast<double>(p.inv_freq[i]) * 0.15915494309189533577;
            float sn, cn;
            sincospif(2.f * static_cast<float>(turns - rint(turns)), &sn, &cn);
            cs[k] = make_float2(cn, sn);
        }
    };
    auto turn = [&](unsigned g, int it, uint4 v0, uint4 v1, const float2 *cs) {
        unsigned b, ti;
        int j, row;
        place(g, it, b, ti, j, row);
        const bool is_q = row < p.Hq, is_v = row >= p.Hq + p.Hkv;
        const float *w = is_q ? p.wq : p.wk;
        float x[16];
        bf16x8_to_f32(v0, x);
        bf16x8_to_f32(v1, x + 8);
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 16; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
        for (int o = 1; o < TPR; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        uint16_t *dst;
        if (is_q) dst = p.q + ((static_cast<long long>(b) * p.n + ti) * p.Hq + row) * D;
        else {
            const int h = row - p.Hq - (is_v ? p.Hkv : 0);
            dst = (is_v ? p.V : p.K) + ((static_cast<long long>(b) * p.Hkv + h) * p.n + ti) * D;
        }
        if (!is_v) {
            if (w) {
                const float r = 1.f / sqrtf(ss * (1.f / D) + p.eps);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    x[e] *= r * w[8 * c0 + e];
                    x[8 + e] *= r * w[8 * c1 + e];
                }
            }
            if (u < rc) {
                const float2 *a = cs + j * half;
                if (p.interleaved) {
#pragma unroll
                    for (int e = 0; e < 16; e += 2) {
                        const float2 f = a[(e < 8 ? c0 : c1) * 4 + (e & 7) / 2];
                        const float xa = x[e], xb = x[e + 1];
                        x[e] = xa * f.x - xb * f.y;
                        x[e + 1] = xb * f.x + xa * f.y;
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float2 f = a[c0 * 8 + e];
                        const float xa = x[e], xb = x[8 + e];
                        x[e] = xa * f.x - xb * f.y;
                        x[8 + e] = xb * f.x + xa * f.y;
                    }
                }
            }
            v0 = f32x8_to_bf16(x);
            v1 = f32x8_to_bf16(x + 8);
        }
        if (it < static_cast<int>(tokens_of(g)) * rows) {
            *reinterpret_cast<uint4 *>(dst + 8 * c0) = v0;
            *reinterpret_cast<uint4 *>(dst + 8 * c1) = v1;
        }
    };
    const unsigned g = blockIdx.x;
    uint4 v0, v1;
    fetch(g, first, v0, v1);
    angles(g, cs_s);
    __syncthreads();
    const int items = static_cast<int>(tokens_of(g)) * rows;
    for (int it0 = 0; it0 < items; it0 += step) {   // (uniform over the CTA)
        uint4 n0 = v0, n1 = v1;
        if (it0 + step < items) fetch(g, it0 + step + first, n0, n1);   // on its way meanwhile
        turn(g, it0 + first, v0, v1, cs_s);
        v0 = n0;
        v1 = n1;
    }
}

}  // namespace

cudaError_t launch_rope(const RopeParams &p, cudaStream_t st) {
    const int rows = p.Hq + 2 * p.Hkv, tpr = p.D / 16;
    const long long tokens = static_cast<long long>(p.B) * p.n;
    int tpc = kRopeThreads / (rows * tpr);
    if (tpc < 1) tpc = 1;
    if (tpc > 16) tpc = 16;
    for (int t = 16; t >= 4; t /= 2)   // (measured: see rope_kernel)
        if (t > tpc && tokens >= 6LL * kSms * t) tpc = t;
    if (tokens < tpc) tpc = static_cast<int>(tokens);
    const int want = (tpc * rows * tpr + 31) / 32 * 32;
    const int threads = want < kRopeThreads ? want : kRopeThreads;
    const unsigned grid = static_cast<unsigned>((tokens + tpc - 1) / tpc);
    const size_t smem = static_cast<size_t>(tpc) * (p.rot / 2) * sizeof(float2);   // at most 8 KB
    cudaError_t e = p.D == 128 ? launch_pdl(rope_kernel<128>, dim3(grid), dim3(threads), smem, st, p, tpc)
                               : launch_pdl(rope_kernel<64>, dim3(grid), dim3(threads), smem, st, p, tpc);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace kvq
