// Reading the packed cache back: tokens [t0, t0 + n) of a layer as bf16 K and V (sm_100a).
//
// value = code * scale + zero (the format's dequantisation; fp32 FMA, rounded once to bf16);
// the open per-channel key group's bf16 keys are copied.  Bound: HBM, mostly the writes (a
// token's K4V2 keys and values are 128 bytes packed and 512 bytes as bf16).  Measured: 8000 tokens of
// 64 (request, kv head) units, K4V2, 65.4 us: 5.0 TB/s, 77% of the measured copy rate.
//
// One warp per (unit, 32-token block).  A lane's packed words are contiguous (the storage
// format's fragments), its codes belong to 8 tokens x D / 4 channel pairs; rows are put
// together in shared memory (16-byte chunks XOR-ed with the row's low bits: no bank
// conflicts on either side) and leave as full rows of 16-byte stores.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kvq_device.cuh"
#include "kvq_internal.h"
#include "kvq_quant.cuh"

namespace kvq {
namespace {

constexpr int kReadWarps = 4;

__device__ __forceinline__ uint32_t bf16x2(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}

template <int BK, int BV, int KM, int D>
__global__ void __launch_bounds__(kReadWarps * 32) read_kernel(const ReadParams p) {
    pdl_enter();
    constexpr int NJ = D / 32, KS = D / 16, CH = D / 8;   // groups, 16-channel steps, 16-byte chunks of a row
    constexpr int REC = unit_bytes(D, BK, BV, KM, 2);
    constexpr int KC = 4 * D * BK, KSZ = 4 * D, VC = 4 * D * BV;
    constexpr int PK = 16 / BK, PV = 16 / BV, WHK = D * BK / 64, WHV = D * BV / 64;
    __shared__ __align__(16) uint8_t rows_s[kReadWarps][32 * D * 2];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const long long item = static_cast<long long>(blockIdx.x) * kReadWarps + warp;
    if (item >= static_cast<long long>(p.B) * p.Hkv * p.nblk) return;   // warps are independent
    const long long unit = item / p.nblk;
    const int blk = p.blk0 + static_cast<int>(item % p.nblk);
    const int b = static_cast<int>(unit / p.Hkv), h = static_cast<int>(unit % p.Hkv);
    const int L = p.len.len(b);
    const int u0 = max(p.t0 - 32 * blk, 0);                        // rows [u0, u1) of the block
    const int u1 = min(min(p.t0 + p.n, L) - 32 * blk, 32);
    if (u1 <= u0) return;
    const uint8_t *rec = p.rec + rec_index(p.btab, b, p.Hkv, h, p.cap_blk, blk) * static_cast<long long>(REC);
    uint8_t *rs = rows_s[warp];
    auto word_at = [&](int u, int chunk, int w) {
        return reinterpret_cast<uint32_t *>(rs + u * (D * 2) + ((chunk ^ (u & 7)) * 16) + w * 4);
    };
    auto flush = [&](uint16_t *out) {   // the warp's rows to out's rows t0 .. of this unit
        __syncwarp();
        uint16_t *o = out + (unit * p.n + 32LL * blk - p.t0) * D;
#pragma unroll
        for (int i = 0; i < 32 * CH / 32; ++i) {
            const int u = (i * 32 + lane) / CH, c = (i * 32 + lane) % CH;
            const uint4 v = *reinterpret_cast<const uint4 *>(rs + u * (D * 2) + ((c ^ (u & 7)) * 16));
            if (u >= u0 && u < u1) *reinterpret_cast<uint4 *>(o + static_cast<long long>(u) * D + 8 * c) = v;
        }
        __syncwarp();
    };
    uint32_t vw[2][WHV];   // loaded up front: on their way while the keys are done
    if (p.V) {
        load_lane_words<WHV>(rec + KC + KSZ, lane, vw[0]);
        load_lane_words<WHV>(rec + KC + KSZ + 2 * D * BV, lane, vw[1]);
    }
    if (p.K) {
        if (KM == 0 && blk == (L >> 5)) {   // the open group: bf16 rows as they are
            const uint16_t *res = p.res + unit * 32 * D;
            uint16_t *o = p.K + (unit * p.n + 32LL * blk - p.t0) * D;
            for (int i = u0 * CH + lane; i < u1 * CH; i += 32)
                *reinterpret_cast<uint4 *>(o + 8LL * i) = *reinterpret_cast<const uint4 *>(res + 8LL * i);
        } else {
            uint32_t kw[2][WHK];
            load_lane_words<WHK>(rec, lane, kw[0]);
            load_lane_words<WHK>(rec + 2 * D * BK, lane, kw[1]);
            if constexpr (KM == 0) {
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    // scale and zero pairs of channels 16k + 2t, +1 and 16k + 8 + 2t, +1
                    const uint4 sz = *reinterpret_cast<const uint4 *>(rec + KC + 16 * (4 * k + t));
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const uint32_t s2 = r ? sz.z : sz.x, z2 = r ? sz.w : sz.y;
#pragma unroll
                        for (int n = 0; n < 4; ++n) {
                            const int slot = (2 * k + (n & 1)) * 2 + r;
                            const uint32_t c2 = unpack<BK>(kw[n >> 1][slot / PK], slot % PK);
                            *word_at(8 * n + g, 2 * k + r, t) =
                                bf16x2(fmaf(half_lo_f(c2), half_lo_f(s2), half_lo_f(z2)),
                                       fmaf(half_hi_f(c2), half_hi_f(s2), half_hi_f(z2)));
                        }
                    }
                }
            } else {
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    const int u = 8 * n + g;
                    float s[NJ], z[NJ];
#pragma unroll
                    for (int j = 0; j < NJ; ++j) {
                        const uint8_t *a = rec + KC + quant::tok_sz_off(u, j, NJ);
                        s[j] = __half2float(*reinterpret_cast<const __half *>(a));
                        z[j] = __half2float(*reinterpret_cast<const __half *>(a + 4 * NJ));
                    }
#pragma unroll
                    for (int k = 0; k < KS; ++k)
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            const int slot = (2 * k + (n & 1)) * 2 + r;
                            const uint32_t c2 = unpack<BK>(kw[n >> 1][slot / PK], slot % PK);
                            *word_at(u, 2 * k + r, t) = bf16x2(fmaf(half_lo_f(c2), s[k / 2], z[k / 2]),
                                                               fmaf(half_hi_f(c2), s[k / 2], z[k / 2]));
                        }
                }
            }
            flush(p.K);
        }
    }
    if (p.V) {
#pragma unroll
        for (int kk = 0; kk < 2; ++kk)
#pragma unroll
            for (int ch = 0; ch < 2; ++ch) {
                const int u = 16 * kk + 8 * ch + 2 * t;   // this lane's token pair
#pragma unroll
                for (int m = 0; m < KS; ++m) {
                    const uint8_t *a = rec + KC + KSZ + VC + quant::tok_sz_off(u, m / 2, NJ);
                    const uint32_t s2 = *reinterpret_cast<const uint32_t *>(a);
                    const uint32_t z2 = *reinterpret_cast<const uint32_t *>(a + 4 * NJ);
#pragma unroll
                    for (int rh = 0; rh < 2; ++rh) {
                        const int slot = 4 * m + 2 * ch + rh;
                        const uint32_t c2 = unpack<BV>(vw[kk][slot / PV], slot % PV);
                        // tokens (u, u + 1) of channel 16m + 8rh + g; with the neighbour channel's
                        // lane: two channels of one token
                        const uint32_t x = bf16x2(fmaf(half_lo_f(c2), half_lo_f(s2), half_lo_f(z2)),
                                                  fmaf(half_hi_f(c2), half_hi_f(s2), half_hi_f(z2)));
                        const uint32_t y = __shfl_xor_sync(0xffffffffu, x, 4);
                        *word_at(u + (g & 1), 2 * m + rh, g >> 1) = (g & 1) ? prmt(y, x, 0x7632) : prmt(x, y, 0x5410);
                    }
                }
            }
        flush(p.V);
    }
}

using ReadFn = void (*)(const ReadParams);

template <int KM, int D>
ReadFn pick_read(int bk, int bv) {
#define KVQ_RCASE(BKv, BVv) \
    if (bk == BKv && bv == BVv) return read_kernel<BKv, BVv, KM, D>;
    KVQ_RCASE(2, 2) KVQ_RCASE(2, 4) KVQ_RCASE(2, 8)
    KVQ_RCASE(4, 2) KVQ_RCASE(4, 4) KVQ_RCASE(4, 8)
    KVQ_RCASE(8, 2) KVQ_RCASE(8, 4) KVQ_RCASE(8, 8)
#undef KVQ_RCASE
    return nullptr;
}

}  // namespace

cudaError_t launch_read(const ReadParams &p, int D, int bk, int bv, int kmode, cudaStream_t st) {
    ReadFn fn = D == 128 ? (kmode == 0 ? pick_read<0, 128>(bk, bv) : pick_read<1, 128>(bk, bv))
                         : (kmode == 0 ? pick_read<0, 64>(bk, bv) : pick_read<1, 64>(bk, bv));
    if (!fn) return cudaErrorInvalidValue;
    const long long items = static_cast<long long>(p.B) * p.Hkv * p.nblk;
    cudaError_t e = launch_pdl(fn, dim3(static_cast<unsigned>((items + kReadWarps - 1) / kReadWarps)),
                               dim3(kReadWarps * 32), 0, st, p);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace kvq
