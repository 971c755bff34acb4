// Attention of several query tokens per request over the packed cache and over the drafted
// tokens themselves (kvq_tree_attn), on the 5th-generation tensor cores (sm_100a).
//
//   s = scale q.k^,  s = cap tanh(s / cap),  s -= slope (pos_q - pos_k);  out = softmax(s) v^
//
// The T * G query rows that share a kv head form row tiles of 128.  A CTA (one per SM) runs a
// part of one unit's keys against its rows.  Roles:
//   warps 0-7   softmax: two slots of 128 threads, a thread per row of the slot's score tile.
//   warps 8-15  unpack: warp 8 + w writes key block w (of 4) of each 128-token tile as fp16
//               code * scale + zero, warp 12 + w the value block.
//   warp 16     issues the MMAs: S = Q K^T (operands in shared memory), O += P V (P in tensor
//               memory over S's last 64 columns).
//   warps 17, 18 issue the bulk copies of the packed key and value parts, a tile's four blocks
//               to a stage.
// While one slot is in its softmax the other's MMAs run.
//
// Rows and slots.  More than 128 rows (TWO): slot j has row tile j, so each packed block is
// unpacked once for up to 256 rows.  Otherwise both slots have the same rows and take the key
// tiles in turn.  Up to 64 or 32 rows fill the 128 lanes as REP = 2 or 4 copies; copy c
// weighs columns [c, c + 1) * 128 / REP of each tile (its other weights are zero), so all
// warps share the softmax.  Slots and copies keep their own m, l and O and are joined at the
// end.
//
// Tiles.  First the "open" ones, keys that are bf16: 32 places for the open per-channel key
// group, if there is one (bf16 residual; its values are packed), then the drafted tokens.  Then
// the whole packed blocks.  Four 32-token blocks to a tile, every operand fp16 in the
// 128-byte-swizzled K-major layout.  The channel order inside a key or query row and the token
// order inside a tile are permuted (both operands of a product alike) so that a lane's
// unpacked pairs are one 16-byte store without bank conflicts:
//   channel d = 64 ks + 32 i + 16 k + 8 r + 2 t + hb  ->  64 ks + 16 t + 8 i + 4 k + 2 r + hb
//   token u of block w: u = 16 kk + 8 ch + 2 t + hb   ->  64 (w / 2) + 16 t + 8 (w % 2) + 4 kk + 2 ch + hb
//
// Measured (Llama shape, 8 kv heads, 4 query heads each): 64 drafted tokens at batch 16, context
// 32768, K4V4: 0.70 ms, 0.79 PFLOP/s, 47% of the measured bf16 rate; 16 drafted tokens at batch
// 64, context 4096, K4V2: 214 us (padded to 128 rows, the MMAs alone would take 63 us, the bytes
// 44 us).  What bounds it.  One row tile (64 rows): the issue of the unpack and softmax warps; the
// tensor pipe is active 30% of the cycles, 47% of issue slots are used, and the stall that leads
// among warps that could run is the instruction fetch (no_instruction, 1.4 cycles per issued
// instruction): four roles share each scheduler's instruction cache, hence small loop bodies
// rather than unrolled ones.  Two row tiles: 39% of issue slots, tensor pipe 27%, XU 27%, so no
// pipe: the handshakes between the roles (waiting roles: 5.5 cycles per issue).  The grid adds to it:
// one split count for all requests, so 128 CTAs leave 20 of 148 SMs idle, 512 take 3.46 waves, and a
// ragged batch ends with its longest request.  A capped score costs two more special-function
// operations (500-token chunks: 132 us capped, 98 us not).  A single short request (11 us, 9.5 us
// with nothing cached): launch, a CTA's set-up, and one pass through the roles.  Registers: the four
// instances without copies spill 64 to 100 bytes, those with two copies 8.
// Measured and not kept: a second team of unpack warps (no gain, slower starts),
// polynomial exponentials for part of a row (4-17% slower: more instructions), a single pass with
// a lagging maximum (slower), four operand buffers with two row tiles (the copies' ring shrinks
// to one stage), unpack loops of their own for open and packed tiles (2-10% slower single requests).
//
// Roundings.  A cached key or value is one fp16 FMA of its exact code: off by 2^-11 of itself
// at most, and exact below fp16's normal numbers (code, scale and zero are whole multiples of
// the step there).  Query rows and bf16 key rows are scaled by a power of two to below 2^15
// (exact in fp16 to 2^-38 of the row's largest); layers with a value that would leave fp16's
// range are scaled down as a whole, by 2^e (e = 1 .. 10; a scale or zero below 2^(e-14) is then
// off by 2^(e-25), so a value by 2^(e+b-25) at most).  Weights are fp16 of 2^(s - m + 7), off by
// 2^-11 (subnormal ones by 2^-32 of the row's largest): m follows the running maximum, and lags
// by up to 2^8 so that the sums in tensor memory are rescaled only when it grew by more; l sums
// them before that rounding.  Scores, m, l and O are fp32.  Drafted values have the whole range
// of bf16, and small ones would be fp16 subnormals or zero: a split's open tiles have an exponent
// of their own (value_exp), and O goes from their unit to the packed tiles' as it does when m
// grows.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <mutex>

#include "kvq_device.cuh"
#include "kvq_internal.h"
#include "kvq_quant.cuh"

namespace kvq {
namespace {

constexpr float kLog2eT = 1.4426950408889634f;
constexpr int kTreeThreads = 20 * 32;    // five warpgroups: register counts are set per warpgroup
// Registers of a thread: 96 at launch (20 warps); the softmax warps hold a whole score row.
// 256 x 144 + 256 x 72 + 128 x 40 = 60,416 of the 640 x 96 = 61,440 launched with.
constexpr int kRegsSoftmax = 144, kRegsUnpack = 72, kRegsIssue = 40;
static_assert(256 * kRegsSoftmax + 256 * kRegsUnpack + 128 * kRegsIssue <= kTreeThreads * 96, "register split");
constexpr int kTile = 128;              // tokens of a key tile, rows of a row tile
constexpr float kWeightBias = 7.f;      // weights are 2^(s - m + 7), s - m <= 8
constexpr float kLag = 8.f;
constexpr uint32_t kTmemCols = 512;     // S0, S1, O0, O1
constexpr int kWeightCol = 64;          // a slot's weights: the last 64 of its 128 score columns

// ------------------------------------------------------------------ tcgen05
// Shared-memory descriptor: K-major, 128-byte swizzle, 8-row groups 1024 bytes apart.
__device__ __forceinline__ uint64_t sw128_desc(uint32_t saddr) {
    return static_cast<uint64_t>((saddr >> 4) & 0x3FFF) | (1ull << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}
// Instruction descriptor of kind::f16: fp16 operands (K-major), fp32 accumulator, M x N.
__host__ __device__ constexpr uint32_t f16_idesc(int M, int N) {
    return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}
// Issued by the lane whose `on` is set.  The predicate is inside the assembly: the code around
// it stays convergent, so the compiler keeps descriptors and addresses in uniform registers (in
// a branch that one lane takes, issuing eight of these took 493 cycles instead of 224, as long
// as they run).
__device__ __forceinline__ void mma_ss(uint32_t on, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"(on)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t on, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(acc), "r"(on)
        : "memory");
}
__device__ __forceinline__ void mma_commit(uint32_t on, uint64_t *bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
        "r"(on)
        : "memory");
}
__device__ __forceinline__ void arrive_one(uint32_t on, uint64_t *bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t@q mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}" ::"r"(
            smem_u32(bar)),
        "r"(on)
        : "memory");
}
__device__ __forceinline__ void expect_one(uint32_t on, uint64_t *bar, uint32_t bytes) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t"
        "@q mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}" ::"r"(smem_u32(bar)),
        "r"(bytes), "r"(on)
        : "memory");
}
__device__ __forceinline__ void bulk_one(uint32_t on, uint32_t dst, const void *src, uint32_t bytes, uint64_t *bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %4, 0;\n\t"
        "@q cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n\t}" ::"r"(dst),
        "l"(src), "r"(bytes), "r"(smem_u32(bar)), "r"(on)
        : "memory");
}
// One lane of a converged warp.
__device__ __forceinline__ uint32_t elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p;
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

#define KVQ_R8(r, o) "+r"(r[o]), "+r"(r[o + 1]), "+r"(r[o + 2]), "+r"(r[o + 3]), "+r"(r[o + 4]), "+r"(r[o + 5]), "+r"(r[o + 6]), "+r"(r[o + 7])
// 32 columns of this warp's 32 lanes, one per register; the registers hold the values after
// ld32_wait on the same array.
__device__ __forceinline__ void ld32_issue(uint32_t taddr, uint32_t *r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void ld32_wait(uint32_t *r) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" : KVQ_R8(r, 0), KVQ_R8(r, 8), KVQ_R8(r, 16), KVQ_R8(r, 24)::"memory");
}
__device__ __forceinline__ void ld16_issue(uint32_t taddr, uint32_t *r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void ld16_wait(uint32_t *r) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" : KVQ_R8(r, 0), KVQ_R8(r, 8)::"memory");
}
__device__ __forceinline__ void st32(uint32_t taddr, const uint32_t *r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::"r"(r[0]),
        "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
        "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]),
        "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
        "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void st16(uint32_t taddr, const uint32_t *r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(r[0]),
        "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
        "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// ------------------------------------------------------------------ shared memory
// Offsets of one CTA's dynamic shared memory (1024-byte aligned base).
template <int D, bool TWO>
struct TreeSmem {
    static constexpr int OPER = kTile * D * 2;                  // one operand tile
    static constexpr int q = 0;                                 // query row tiles
    static constexpr int kv = q + (TWO ? 2 : 1) * OPER;         // key tiles, value tiles [D channels][128 tokens]
    static constexpr int rowscale = kv + (TWO ? 3 : 4) * OPER;  // score scale of each query row [256]
    // open tiles: key row scales and positions, [4][128] each (tile i uses stage i % 4: when its
    // keys are written, tile i - 2's scores are done, so tile i - 4's softmax is)
    static constexpr int kscale = rowscale + 256 * 4;
    static constexpr int kpos = kscale + 4 * kTile * 4;
    static constexpr int bars = kpos + 4 * kTile * 4;           // barriers, TMEM address, flags
    static constexpr int ring = bars + 512;                     // packed parts
    // the end: (m, l) of the 256 softmax threads over the row scales .. positions, and their O
    // rows (D + 4 floats) over the operand tiles
    static constexpr int ml = rowscale;
    static constexpr int ROW = D + 4;
    static_assert(256 * ROW * 4 <= rowscale && ml + 256 * 8 <= bars, "the joining areas fit");
};

// Operand buffer of the key (v = 0) or value (v = 1) tile of tile i, and how often it was used
// before.  One row tile: two buffers for keys, two for values (keys are scored two tiles
// ahead).  TWO: three buffers in the order of use, K0 V0 K1 V1 ..
template <bool TWO>
__device__ __forceinline__ void operand_buffer(int v, int i, int &buf, int &use) {
    if constexpr (TWO) {
        use = (2 * i + v) / 3;
        buf = 2 * i + v - 3 * use;
    } else {
        use = i >> 1;
        buf = 2 * v + (i & 1);
    }
}

struct TreeBars {
    uint64_t q_full, full[4], free[4], s_full[2], p_full[2], o_full[2];
    uint64_t part_full[2][4], part_free[2][4];   // packed parts (keys, values), per stage
    uint64_t v_ready;      // open_top is final
    uint32_t tmem, bad_value;
    int min_pos;
    uint32_t open_top;     // largest finite |value| of the split's open tiles (float bits; see value_exp)
};
static_assert(sizeof(TreeBars) <= 512, "barrier area");

// Token of column `col` of a tile, and the column of token u of block w.
__host__ __device__ constexpr int tile_token(int col) {
    return 32 * (2 * (col >> 6) + ((col >> 3) & 1)) + 16 * ((col >> 2) & 1) + 8 * ((col >> 1) & 1) + 2 * ((col >> 4) & 3) +
           (col & 1);
}
__host__ __device__ constexpr int tile_col(int w, int u) {
    return 64 * (w >> 1) + 16 * ((u >> 1) & 3) + 8 * (w & 1) + 4 * (u >> 4) + 2 * ((u >> 3) & 1) + (u & 1);
}

__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
__device__ __forceinline__ uint64_t pack2(float a, float b) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ void unpack2(uint64_t v, float &a, float &b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

__device__ __forceinline__ uint32_t hfma2_bits(uint32_t c, uint32_t s, uint32_t z) {
    return h2_bits(__hfma2(bits_h2(c), bits_h2(s), bits_h2(z)));
}
// W consecutive words (4, 2 or 1) of shared memory.
template <int W>
__device__ __forceinline__ void lds_words(uint32_t addr, uint32_t *w) {
    if constexpr (W == 4) {
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(addr));
    } else if constexpr (W == 2) {
        asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr));
    } else {
        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w[0]) : "r"(addr));
    }
}
// A part's scales and zeros (2 D halves at sz, in shared memory) times f, a power of two: by the warp
// that unpacks the part, before it does.  A loop over few words rather than a second instance of
// the unpackers: that one's code beside the others' cost 17% at batch 16, context 32768.
template <int D>
__device__ __forceinline__ void scale_part(uint32_t sz, int lane, float f) {
#pragma unroll 1
    for (int i = lane; i < D; i += 32) {
        uint32_t w;
        lds_words<1>(sz + 4 * i, &w);
        asm volatile("st.shared.b32 [%0], %1;" ::"r"(sz + 4 * i), "r"(pack_h2(half_lo_f(w) * f, half_hi_f(w) * f)) : "memory");
    }
    __syncwarp();
}
// Byte offset, within a half's code area, of a lane's words [BITS / 2 * i, ..) : the words of
// eight consecutive slots (a 32-channel step of keys, a channel group of values).
template <int BITS, int D>
__device__ __forceinline__ int step_words(int i, int lane) {
    constexpr int WH = D * BITS / 64, C = WH < 4 ? WH : 4, W = BITS / 2;   // words of a half, chunk, of a step
    const int w = W * i;
    return ((w / C) * 32 * C + lane * C + w % C) * 4;
}

// Key block w of a tile (part: [codes][s/z] in shared memory) -> fp16 rows of the K operand.
// A loop step covers the 32 channels of one 16-byte chunk index; it is not
// unrolled: four copies of the step's code do not fit the instruction caches beside the other
// roles'.
template <int BK, int KM, int D>
__device__ __forceinline__ void unpack_keys(const uint8_t *part, uint8_t *kt, int w, int lane) {
    constexpr int NJ = D / 32, PK = 16 / BK, KC = 4 * D * BK, W = BK / 2;
    const int g = lane >> 2, t = lane & 3;
    const uint32_t ps = smem_u32(part);
    // row of token u = 16 kk + 8 i + g, n = 2 kk + i: row0 + 4 kk + 2 i; its 16-byte chunk
    // 2 t + i2 is XOR-ed with the row's low bits (g & 1) + 4 kk + 2 i: all but the lane's own
    // part is constant
    const uint32_t at0 = smem_u32(kt) + tile_col(w, g) * 128 + (((2 * t) ^ (g & 1)) << 4);
#pragma unroll 1
    for (int i = 0; i < D / 32; ++i) {   // channels 32 i ..: chunk i2 = i % 2 of sub-tile i / 2
        const uint32_t at = (at0 ^ ((i & 1) << 4)) + (i >> 1) * (kTile * 128);
        uint32_t kw[2][W], s[2][2], z[2][2];
        lds_words<W>(ps + step_words<BK, D>(i, lane), kw[0]);
        lds_words<W>(ps + 2 * D * BK + step_words<BK, D>(i, lane), kw[1]);
        if constexpr (KM == 0) {
#pragma unroll
            for (int k1 = 0; k1 < 2; ++k1) {   // scale and zero pairs of channels 32 i + 16 k1 + 8 r + 2 t, +1
                uint32_t a[4];
                lds_words<4>(ps + KC + 16 * (4 * (2 * i + k1) + t), a);
                s[k1][0] = a[0]; z[k1][0] = a[1]; s[k1][1] = a[2]; z[k1][1] = a[3];
            }
        }
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            uint32_t st = 0, zt = 0;
            if constexpr (KM == 1) {   // scale of (token, 32-channel group i)
                const uint8_t *a = part + KC + quant::tok_sz_off(8 * n + g, i, NJ);
                st = *reinterpret_cast<const uint16_t *>(a) * 0x10001u;
                zt = *reinterpret_cast<const uint16_t *>(a + 4 * NJ) * 0x10001u;
            }
            uint32_t o[4];
#pragma unroll
            for (int k1 = 0; k1 < 2; ++k1)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const int slot = (2 * k1 + (n & 1)) * 2 + r;   // of the step's eight
                    const uint32_t c2 = unpack<BK>(kw[n >> 1][slot / PK], slot % PK);
                    o[2 * k1 + r] = KM == 0 ? hfma2_bits(c2, s[k1][r], z[k1][r]) : hfma2_bits(c2, st, zt);
                }
            const int low = 4 * (n >> 1) + 2 * (n & 1);
            sts128((at ^ (low << 4)) + low * 128, o[0], o[1], o[2], o[3]);
        }
    }
}

// Value block w of a tile -> fp16 columns of the V operand ([channel][token]); tokens from
// `valid` on become zeros.  A loop step covers one 32-channel group.
template <int BV, int D>
__device__ __forceinline__ void unpack_values(const uint8_t *part, uint8_t *vt, int w, int lane, int valid) {
    constexpr int NJ = D / 32, PV = 16 / BV, VC = 4 * D * BV, W = BV / 2;
    const int g = lane >> 2, t = lane & 3;
    const uint32_t ps = smem_u32(part);
    const uint32_t base = smem_u32(vt) + (w >> 1) * (D * 128) + g * 128 + (((2 * t + (w & 1)) ^ g) << 4);
#pragma unroll 1
    for (int j = 0; j < NJ; ++j) {
        uint32_t vw[2][W], s[4], z[4];
        lds_words<W>(ps + step_words<BV, D>(j, lane), vw[0]);
        lds_words<W>(ps + 2 * D * BV + step_words<BV, D>(j, lane), vw[1]);
#pragma unroll
        for (int n = 0; n < 4; ++n) {   // token pair 8 n + 2 t, +1
            lds_words<1>(ps + VC + quant::tok_sz_off(8 * n + 2 * t, j, NJ), &s[n]);
            lds_words<1>(ps + VC + quant::tok_sz_off(8 * n + 2 * t, j, NJ) + 4 * NJ, &z[n]);
        }
        if (valid < 32) {   // the unused tokens' scales are not written: they may hold anything
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                const int u = 8 * n + 2 * t;
                const uint32_t m = (u < valid ? 0xFFFFu : 0u) | (u + 1 < valid ? 0xFFFF0000u : 0u);
                s[n] &= m;
                z[n] &= m;
            }
        }
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int rh = 0; rh < 2; ++rh) {
                uint32_t o[4];
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    const int slot = 4 * m + 2 * (n & 1) + rh;
                    o[n] = hfma2_bits(unpack<BV>(vw[n >> 1][slot / PV], slot % PV), s[n], z[n]);
                }
                sts128(base + j * (32 * 128) + (16 * m + 8 * rh) * 128, o[0], o[1], o[2], o[3]);
            }
    }
}

// The unpackers by bit width.
template <int KM, int D>
__device__ __forceinline__ void unpack_keys_bits(int bits, const uint8_t *part, uint8_t *kt, int w, int lane) {
    if (bits == 8) unpack_keys<8, KM, D>(part, kt, w, lane);
    else if (bits == 4) unpack_keys<4, KM, D>(part, kt, w, lane);
    else unpack_keys<2, KM, D>(part, kt, w, lane);
}
template <int D>
__device__ __forceinline__ void unpack_values_bits(int bits, const uint8_t *part, uint8_t *vt, int w, int lane, int valid) {
    if (bits == 8) unpack_values<8, D>(part, vt, w, lane, valid);
    else if (bits == 4) unpack_values<4, D>(part, vt, w, lane, valid);
    else unpack_values<2, D>(part, vt, w, lane, valid);
}

// Byte offset of channel chunk c8 (8 channels d = 8 c8 ..) of `row` in a K-major operand whose
// channels are permuted: the chunk's pair t goes to word 4 t' of the row (see the top); this is
// the offset of pair 0, pair t is 32 bytes of row further before the swizzle.
__device__ __forceinline__ int permuted_pair(int row, int c8, int t) {
    // d = 8 c8 + 2 t: ks = c8 / 8, i = (c8 / 4) % 2, k = (c8 / 2) % 2, r = c8 % 2
    const int chunk = 2 * t + ((c8 >> 2) & 1);
    return (c8 >> 3) * (kTile * 128) + row * 128 + ((chunk ^ (row & 7)) << 4) + ((c8 >> 1) & 1) * 8 + (c8 & 1) * 4;
}

// Row of 8 * NL channels held by NL lanes (8 bf16 channels each): scaled by a power of two to
// a largest magnitude in [2^14, 2^15) and written as fp16; returns the inverse scale.
template <int NL>
__device__ __forceinline__ float store_scaled_row(uint8_t *tile, int row, int c8, const uint4 &x, float sign) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    float f[8], mx = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        mx = fmaxf(mx, fmaxf(fabsf(f[2 * i]), fabsf(f[2 * i + 1])));
    }
#pragma unroll
    for (int o = 1; o < NL; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    // exponent of the largest (kept above -112 so that the inverse scale is a normal number);
    // two exact factors, since the values are first scaled to about one
    const int e = mx > 0.f ? max(-112, min(127, floor_log2(mx))) : 14;
    const int a = (14 - e) / 2, b = 14 - e - a;
    const float fa = pow2f(a) * sign, fb = pow2f(b);
#pragma unroll
    for (int t = 0; t < 4; ++t)
        *reinterpret_cast<uint32_t *>(tile + permuted_pair(row, c8, t)) =
            h2_bits(__floats2half2_rn(f[2 * t] * fa * fb, f[2 * t + 1] * fa * fb));
    return pow2f(e - 14);
}

// Exponent e of the power of two that the values of a split's open tiles are divided by, from their
// largest magnitude: the packed tiles' ev unless that is below 2^(ev - 3), else the one that brings
// it to [2^14, 2^15).  So a value is off by 2^-11 of itself or 2^-22 of the largest, whichever is
// more, and values of ordinary size share the packed tiles' exponent (no rescale between them).
constexpr int kMinValueExp = -112;   // (2^-e stays a normal number)
__device__ __forceinline__ int value_exp(uint32_t top_bits, int ev) {
    const float top = __uint_as_float(top_bits);
    return top >= pow2f(ev - 3) ? ev : max(kMinValueExp, floor_log2(top) - 14);   // (0: the least)
}

// Bounded waits; after one expiry no wait waits again.  The clock is read only after many
// polls: reading the global timer takes longer than most of these waits.
struct Waiter {
    bool failed = false;
    __device__ __forceinline__ void operator()(uint64_t *bar, unsigned parity) {
        if (mbar_try_wait(bar, parity)) return;
        slow(bar, parity);
    }
    __device__ __forceinline__ void slow(uint64_t *bar, unsigned parity) {
        if (failed) return;
        uint64_t t0 = 0;
        for (;;) {
#pragma unroll 1
            for (int k = 0; k < 256; ++k)
                if (mbar_try_wait(bar, parity)) return;
            const uint64_t t = globaltimer_ns();
            if (t0 == 0) t0 = t;
            if (t - t0 > kWaitLimitNs) break;
        }
        failed = true;
    }
};

// ------------------------------------------------------------------ kernel
template <int D, bool TWO, int REP>
__global__ void __launch_bounds__(kTreeThreads, 1) tree_kernel(const __grid_constant__ TreeParams p) {
    pdl_enter();
    using SM = TreeSmem<D, TWO>;
    constexpr int NL = D / 8;                                 // 8-channel chunks of a row
    constexpr int COPY = kTile / REP;                         // query rows of a score tile
    constexpr int ROWS = TWO ? 256 : COPY;                    // query rows of the CTA
    constexpr int NC = 4 / REP;                               // 32-column chunks that a row weighs
    static_assert(!TWO || REP == 1, "two row tiles have no copies");
    extern __shared__ __align__(1024) uint8_t smem[];
    TreeBars *bar = reinterpret_cast<TreeBars *>(smem + SM::bars);
    float *rowscale = reinterpret_cast<float *>(smem + SM::rowscale);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int sp = blockIdx.x, b = blockIdx.z;
    const int groups = gridDim.y / p.Hkv, h = blockIdx.y / groups, rg = blockIdx.y % groups;
    const int row0 = rg * ROWS;                               // first query row (t G + g) of this CTA
    const int nq = p.len.queries(b), L = p.len.len(b);
    const int nrow = min(ROWS, nq * p.G - row0);              // live rows
    if (nrow <= 0) return;
    const int Hq = p.Hkv * p.G;
    const long long unit = static_cast<long long>(b) * p.Hkv + h;
    const unsigned top_k = p.top[0], top_v = p.top[1];
    const int *depth = p.depth ? p.depth + static_cast<long long>(b) * p.T : nullptr;
    auto row_t = [&](int r) { return p.gmul ? static_cast<int>(__umulhi(row0 + r, p.gmul)) : row0 + r; };   // / G

    if (warp == 17) {   // a barrier per lane: 15 of the operand tiles, 16 of the packed parts
        if (lane < 15) {   // q_full, full, free, s_full, p_full, o_full
            mbar_init(&bar->q_full + lane, lane == 0 ? 8 : (lane < 5 || lane == 11 || lane == 12 ? 4 : 1));
        } else if (lane < 31) {
            mbar_init(&bar->part_full[0][0] + (lane - 15), lane < 23 ? 1 : 4);
        } else {
            bar->bad_value = 0;
            bar->min_pos = 0x7FFFFFFF;
            bar->open_top = 0;
            mbar_init(&bar->v_ready, 4);
        }
        fence_mbar_init();
    }
    if (warp == 16) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&bar->tmem)),
                     "r"(kTmemCols));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = bar->tmem;
    // query positions; the earliest one's window bounds the tiles
    auto query_pos = [&](int r) { return L + (depth ? depth[row_t(r)] : row_t(r)); };
    if (p.window) {
        if (tid < nrow) atomicMin(&bar->min_pos, query_pos(tid));
        __syncthreads();
    }
    // open keys: places for the open key group, then drafted tokens (a chunk: those up to the
    // last row)
    const int open = p.kmode == 0 ? L & 31 : 0, pad = open ? 32 : 0;
    const int nk = p.mask ? nq : min(nq, row_t(nrow - 1) + 1);
    const int n_open = (pad + nk + kTile - 1) / kTile;
    const int nblk = (L - open + 31) >> 5;                    // packed blocks
    int tile_first = 0;
    if (p.window) {
        const long long lo = static_cast<long long>(bar->min_pos) - p.window + 1;
        if (lo > 0) tile_first = static_cast<int>(min(lo, static_cast<long long>(L)) / kTile);
    }
    const int n_main = max(0, (nblk + 3) / 4 - tile_first);
    // this split's even part of the tiles: [tb, te), open tiles first
    const int n_all = n_open + n_main;
    // (at most 2^23 tiles and 64 splits: 32 bits)
    const int tb = static_cast<unsigned>(n_all) * sp / static_cast<unsigned>(p.S);
    const int te = static_cast<unsigned>(n_all) * (sp + 1) / static_cast<unsigned>(p.S);
    const int n = te - tb;
    Waiter wait;

    // exponent of the power of two that the layer's cached values are divided by: 0 unless a group's
    // bound is above fp16's range (finite scales and zeros: below 2^24 + 2^16, so 10 at most)
    auto pre_exp = [](unsigned top) { return top ? min(10, floor_log2(__uint_as_float(top)) - 14) : 0; };
    const int ek = pre_exp(top_k), ev = pre_exp(top_v);

    // packed parts: first block and number of blocks of tile tb + i (the open group has packed
    // values only); bytes, ring
    const int key_part = 4 * D * p.bk + 4 * D, value_part = 4 * D * p.bv + 4 * D;
    auto blocks_of = [&](bool is_v, int i, int &blk0) {
        const int ti = tb + i - n_open;
        if (ti < 0) {
            blk0 = L >> 5;
            return is_v && pad && tb + i == 0 ? 1 : 0;
        }
        blk0 = 4 * (tile_first + ti);
        return min(4, nblk - blk0);
    };
    auto ring_of = [&](bool is_v) { return smem + SM::ring + (is_v ? 4 * p.dk * key_part : 0); };

    if (warp >= 8 && warp < 16) {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsUnpack));
      if (n > 0) {
        // ================================================================ unpack warps
        const int w8 = warp - 8, w = w8 & 3;
        const bool is_v = w8 >= 4;
        const int bits = is_v ? p.bv : p.bk;
        const int part_bytes = is_v ? value_part : key_part;
        const int stages = is_v ? p.dv : p.dk;
        const uint8_t *ring = ring_of(is_v) + w * part_bytes;
        const uint32_t on = elect_one();
        int vexp = ev;             // exponent of the open tiles' values
        if (is_v && tb < n_open) {
            // Largest finite magnitude of the split's drafted values and of the open group's.  A warp
            // stops at the first value that leaves the exponent at ev: for ordinary values after one
            // load.
            const int ja = max(0, kTile * tb - pad), je = min(nk, kTile * min(te, n_open) - pad);
            const uint4 *v = reinterpret_cast<const uint4 *>(p.vd + (unit * p.T + ja) * D);
            const float enough = pow2f(ev - 3);
            float top = 0.f;
            for (int it = 32 * w + lane, end = (je - ja) * NL; it - lane < end; it += 128) {
                const uint4 x = it < end ? v[it] : make_uint4(0u, 0u, 0u, 0u);
                const uint32_t xw[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float a = fabsf(__uint_as_float(k & 1 ? xw[k >> 1] & 0xFFFF0000u : xw[k >> 1] << 16));
                    if (a < INFINITY) top = fmaxf(top, a);
                }
                if (__any_sync(0xffffffffu, top >= enough)) break;
            }
            if (w == 0 && pad && tb == 0 && !__any_sync(0xffffffffu, top >= enough)) {
                // the open group's packed values: a bound, |zero| + scale (2^b - 1), per token
                const uint8_t *sz = p.rec + (rec_index(p.btab, b, p.Hkv, h, p.cap_blk, L >> 5) + 1) * (key_part + value_part) - 4 * D;
                for (int j = 0; lane < open && j < NL / 4; ++j) {
                    const uint8_t *a = sz + quant::tok_sz_off(lane, j, NL / 4);
                    const float sc = __half2float(*reinterpret_cast<const __half *>(a));
                    const float ze = __half2float(*reinterpret_cast<const __half *>(a + NL));
                    top = fmaxf(top, fmaf(sc, static_cast<float>((1 << bits) - 1), fabsf(ze)));
                }
            }
            const uint32_t wtop = __reduce_max_sync(0xffffffffu, __float_as_uint(top));
            if (on) atomicMax(&bar->open_top, wtop);
            __syncwarp();
            arrive_one(on, &bar->v_ready);
            wait(&bar->v_ready, 0);
            vexp = value_exp(bar->open_top, ev);
        }
        int st = 0, ph = 0;        // the next part's stage and phase (tiles without a part use none)
        for (int i = 0; i < n; ++i) {
            int buf, used;
            operand_buffer<TWO>(is_v, i, buf, used);
            uint8_t *tile = smem + SM::kv + buf * SM::OPER;
            int blk;
            const int nb = blocks_of(is_v, i, blk);
            const bool has = w < nb;                          // this warp's block is packed
            blk += w;
            // a warp without a block waits too: its next wait must not meet this phase unfinished
            if (nb > 0) wait(&bar->part_full[is_v][st], ph);
            if (used > 0) wait(&bar->free[buf], (used - 1) & 1);
            const uint8_t *part = ring + st * 4 * part_bytes;
            const bool is_open = tb + i < n_open;
            const int ex = !is_v ? ek : (is_open ? vexp : ev);
            if (ex != 0 && has) scale_part<D>(smem_u32(part) + part_bytes - 4 * D, lane, pow2f(-ex));
            const int j0 = kTile * (tb + i) + 32 * w - pad;   // open tiles: the block's first drafted token
            if (!is_v && has) {
                if (p.kmode == 0) unpack_keys_bits<0, D>(bits, part, tile, w, lane);
                else unpack_keys_bits<1, D>(bits, part, tile, w, lane);
            } else if (!is_v && is_open) {
                // bf16 rows: the open group's, or drafted tokens (rows behind them are masked)
                float *ksc = reinterpret_cast<float *>(smem + SM::kscale) + (i & 3) * kTile;
                int *kp = reinterpret_cast<int *>(smem + SM::kpos) + (i & 3) * kTile;
                constexpr int RPW = 32 / NL, BATCH = 4;
                const int c8 = lane % NL;
                const int rows = j0 < 0 ? open : min(32, nk - j0);
                const uint16_t *k0 = j0 < 0 ? p.res + unit * 32 * D : p.kd + (unit * p.T + j0) * D;
#pragma unroll 1
                for (int u0 = 0; u0 < rows; u0 += RPW * BATCH) {
                    uint4 x[BATCH];
#pragma unroll
                    for (int k = 0; k < BATCH; ++k) {
                        const int u = u0 + k * RPW + lane / NL;
                        x[k] = make_uint4(0u, 0u, 0u, 0u);
                        if (u < rows) x[k] = *reinterpret_cast<const uint4 *>(k0 + u * D + 8 * c8);
                    }
#pragma unroll
                    for (int k = 0; k < BATCH; ++k) {
                        const int u = u0 + k * RPW + lane / NL, row = tile_col(w, u);
                        const float inv = store_scaled_row<NL>(tile, row, c8, x[k], 1.f);
                        if (c8 == 0) ksc[row] = inv * pow2f(-ek);   // the row scale carries 2^ek for the cached keys
                    }
                }
                if (p.alibi || p.window)   // key positions (only these read them)
                    kp[tile_col(w, lane)] =
                        j0 < 0 ? (L & ~31) + lane : (lane < rows ? L + (depth ? depth[j0 + lane] : j0 + lane) : 0);
            } else if (is_v && has) {
                const int valid = min(32, L - 32 * blk);
                unpack_values_bits<D>(bits, part, tile, w, lane, valid);
            } else if (is_v && is_open && j0 < nk) {
                // drafted values: token pairs (u, u + 1) of the block
                const float fs = pow2f(-vexp);
                bool bad = false;
                for (int it = lane; it < 16 * NL; it += 32) {
                    const int u = 2 * (it % 16), c = 8 * (it / 16), col = tile_col(w, u);
                    float f[2][8];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        uint4 x = make_uint4(0u, 0u, 0u, 0u);
                        if (j0 + u + e < nk) x = *reinterpret_cast<const uint4 *>(p.vd + (unit * p.T + j0 + u + e) * D + c);
                        const uint32_t xw[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            float v = __uint_as_float(k & 1 ? xw[k >> 1] & 0xFFFF0000u : xw[k >> 1] << 16);
                            // a weight of zero must not meet NaN or infinity: those are added in
                            // the end, to the rows that see them
                            if (!(fabsf(v) < INFINITY)) { bad = true; v = 0.f; }
                            f[e][k] = fminf(fmaxf(v * fs, -65504.f), 65504.f);
                        }
                    }
                    uint8_t *at = tile + (col >> 6) * (D * 128) + c * 128 + (col & 7) * 2;
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        *reinterpret_cast<uint32_t *>(at + k * 128 + ((((col & 63) >> 3) ^ k) << 4)) =
                            h2_bits(__floats2half2_rn(f[0][k], f[1][k]));
                }
                if (bad) bar->bad_value = 1;
            } else if (is_v) {   // nothing here: the weights are zero, the values must be finite
                const int g = lane >> 2, t = lane & 3;
                const uint32_t at = smem_u32(tile) + (w >> 1) * (D * 128) + g * 128 + (((2 * t + (w & 1)) ^ g) << 4);
                for (int c = 0; c < D; c += 8) sts128(at + c * 128, 0u, 0u, 0u, 0u);
            }
            fence_proxy_async();
            __syncwarp();
            arrive_one(on, &bar->full[buf]);
            if (nb > 0) {
                arrive_one(on, &bar->part_free[is_v][st]);
                if (++st == stages) st = 0, ph ^= 1;
            }
        }
      }
    } else if (warp >= 16) {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsIssue));
      if (warp == 17 || warp == 18) {
        // ================================================================ packed parts
        const bool is_v = warp == 18;
        const int stages = is_v ? p.dv : p.dk, bytes = is_v ? value_part : key_part;
        const long long rec_bytes = key_part + value_part;
        const uint8_t *src = p.rec + (is_v ? key_part : 0);
        const uint32_t ring = smem_u32(ring_of(is_v)), on = elect_one();
        bool lap = false;      // every stage has been used
        int st = 0, ph = 0;
        for (int i = 0; i < n; ++i) {
            int blk0;
            const int nb = blocks_of(is_v, i, blk0);
            if (nb <= 0) continue;
            if (lap) wait(&bar->part_free[is_v][st], ph ^ 1);
            __syncwarp();
            expect_one(on, &bar->part_full[is_v][st], nb * bytes);
#pragma unroll
            for (int w = 0; w < 4; ++w)
                if (w < nb)
                    bulk_one(on, ring + (st * 4 + w) * bytes,
                             src + rec_index(p.btab, b, p.Hkv, h, p.cap_blk, blk0 + w) * rec_bytes, bytes,
                             &bar->part_full[is_v][st]);
            if (++st == stages) st = 0, ph ^= 1, lap = true;
        }
        // no copy is in flight when the CTA ends, whatever wait expired before: each used stage's
        // last phase (stages below st were filled in this lap, the others in the one before)
        Waiter drain;
        for (int k = 0; k < (lap ? stages : st); ++k) drain(&bar->part_full[is_v][k], k < st ? ph : ph ^ 1);
        wait.failed |= drain.failed;
      } else if (warp == 16 && n > 0) {
        // ================================================================ MMA issue
        {
            const uint32_t on = elect_one();
            constexpr uint32_t IQK = f16_idesc(128, kTile), IPV = f16_idesc(128, D);
            constexpr int STEP = TWO ? 1 : 2;   // tiles from a slot's tile to its next
            wait(&bar->q_full, 0);
            auto qk = [&](int j, int i) {
                const uint64_t a = sw128_desc(smem_u32(smem + SM::q + (TWO ? j * SM::OPER : 0)));
                int buf, used;
                operand_buffer<TWO>(0, i, buf, used);
                const uint64_t k = sw128_desc(smem_u32(smem + SM::kv + buf * SM::OPER));
                if (!TWO || j == 0) wait(&bar->full[buf], used & 1);
                fence_after();
                __syncwarp();
#pragma unroll
                for (int s = 0; s < D / 16; ++s) {   // 16 channels: 32 bytes on, 64 channels: the next sub-tile
                    const int off = ((s >> 2) * (kTile * 128) + (s & 3) * 32) >> 4;
                    mma_ss(on, tmem + j * 128, a + off, k + off, IQK, s > 0);
                }
                mma_commit(on, &bar->s_full[j]);
                if (!TWO || j == 1) mma_commit(on, &bar->free[buf]);
            };
            auto pv = [&](int j, int i, int use, bool last) {
                int buf, used;
                operand_buffer<TWO>(1, i, buf, used);
                const uint64_t v = sw128_desc(smem_u32(smem + SM::kv + buf * SM::OPER));
                if (!TWO || j == 0) wait(&bar->full[buf], used & 1);
                wait(&bar->p_full[j], use & 1);
                fence_after();
                __syncwarp();
#pragma unroll
                for (int s = 0; s < kTile / 16; ++s)
                    mma_ts(on, tmem + 256 + j * 128, tmem + j * 128 + kWeightCol + 8 * s,
                           v + (((s >> 2) * (D * 128) + (s & 3) * 32) >> 4), IPV, (use > 0 || s > 0) ? 1u : 0u);
                if (!TWO || j == 1) mma_commit(on, &bar->free[buf]);
                if (last) mma_commit(on, &bar->o_full[j]);
            };
            // MMAs of one thread run in order: a slot's next scores may overwrite the weights
            // that its previous product reads
            qk(0, 0);
            if (TWO) qk(1, 0);
            else if (n > 1) qk(1, 1);
            for (int i = 0; i < n; ++i)
#pragma unroll 1   // (4% at batch 16, context 32768: the loops' code is what the instruction caches hold)
                for (int j = TWO ? 0 : i & 1; j < (TWO ? 2 : (i & 1) + 1); ++j) {
                    pv(j, i, i / STEP, i + STEP >= n);
                    if (i + STEP < n) qk(j, i + STEP);
                }
            // nor is an MMA in flight when tensor memory is freed
            Waiter drain;
            drain(&bar->o_full[0], 0);
            if (TWO || n > 1) drain(&bar->o_full[1], 0);
            wait.failed |= drain.failed;
        }
        __syncwarp();
      }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
        // ================================================================ softmax
        const uint32_t on = elect_one();
        const int j = warp >> 2;                                 // slot
        const int r = TWO ? tid : (tid & 127) % COPY;            // query row of the CTA
        const int copy = TWO ? 0 : (tid & 127) / COPY;
        const bool busy = (r & ~31) < nrow;                      // the warp has a live row
        const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
        const uint32_t ts = tmem + lanes + j * 128, to = tmem + lanes + 256 + j * 128;
        const int rc = min(r, nrow - 1);                         // dead rows follow a live one
        const int t = row_t(rc), hq = h * p.G + (row0 + rc) - t * p.G;
        const int pos = query_pos(rc);
        const float slope2 = p.alibi ? p.alibi[hq] * kLog2eT : 0.f;
        const uint32_t *mrow = p.mask ? p.mask + (static_cast<long long>(b) * p.T + t) * p.mask_words : nullptr;
        if (n > 0) {   // query rows, REP copies of them; a warp takes RPW rows per step, four steps' loads first
            constexpr int RPW = 32 / NL, STEPS = ROWS / (8 * RPW), BATCH = STEPS < 4 ? STEPS : 4;
            const float sign = p.scale < 0.f ? -1.f : 1.f;
            const float base = fabsf(p.scale) * kLog2eT * pow2f(ek);
            const int c8 = lane % NL;
            const uint16_t *q0 = p.q + (static_cast<long long>(b) * p.T * Hq + h * p.G) * D + 8 * c8;
#pragma unroll 1
            for (int s0 = 0; s0 < STEPS; s0 += BATCH) {
                uint4 x[BATCH];
#pragma unroll
                for (int k = 0; k < BATCH; ++k) {
                    const int r = (8 * (s0 + k) + warp) * RPW + lane / NL;
                    x[k] = make_uint4(0u, 0u, 0u, 0u);
                    if (r < nrow) {
                        const int t = row_t(r), g = (row0 + r) - t * p.G;
                        x[k] = *reinterpret_cast<const uint4 *>(q0 + (static_cast<long long>(t) * Hq + g) * D);
                    }
                }
#pragma unroll
                for (int k = 0; k < BATCH; ++k) {
                    const int r = (8 * (s0 + k) + warp) * RPW + lane / NL;
                    float inv = 1.f;
#pragma unroll
                    for (int cp = 0; cp < REP; ++cp)
                        inv = store_scaled_row<NL>(smem + SM::q + (r >> 7) * SM::OPER, (r & 127) + cp * COPY, c8, x[k], sign);
                    if (c8 == 0) rowscale[r] = base * inv;
                }
            }
            fence_proxy_async();
            __syncwarp();
            arrive_one(on, &bar->q_full);
        }
        // exponent of the open tiles' values (final once the slot's first open tile's values are there)
        auto open_exp = [&]() { return value_exp(bar->open_top, ev); };
        float m = -INFINITY, l = 0.f, rs = 0.f;
        const int first = TWO ? 0 : j, step = TWO ? 1 : 2;
        int use = 0;
        for (int i = first; i < n; i += step, ++use) {
            const int ti = tb + i - n_open;
            const bool is_open = ti < 0;
            const int base = is_open ? kTile * (tb + i) : kTile * (tile_first + ti);   // first place of the tile
            wait(&bar->s_full[j], use & 1);
            fence_after();
            if (use == 0) {
                wait(&bar->q_full, 0);
                rs = rowscale[r];
            }
            if (busy) {
                // the row's visible keys of a packed tile are tokens [lo, hi) of it
                const int hi = min(L - open - base, kTile);
                int lo = 0;
                if (p.window) {
                    const long long x = static_cast<long long>(pos) - p.window + 1 - base;
                    lo = static_cast<int>(max(0LL, min(x, static_cast<long long>(kTile))));
                }
                const bool cut = !is_open && __any_sync(0xffffffffu, lo > 0 || hi < kTile);
                const bool shaped = is_open || p.cap > 0.f || p.alibi || cut;
                // raw scores of chunk c -> log2 units, capped, biased, masked
                auto shape = [&](uint32_t *x, int c) {
                    if (is_open) {
                        const float4 *ksc = reinterpret_cast<const float4 *>(smem + SM::kscale) + ((i & 3) * kTile + 32 * c) / 4;
#pragma unroll
                        for (int e = 0; e < 32; e += 4) {
                            const float4 k4 = ksc[e / 4];
                            x[e] = __float_as_uint(__uint_as_float(x[e]) * (rs * k4.x));
                            x[e + 1] = __float_as_uint(__uint_as_float(x[e + 1]) * (rs * k4.y));
                            x[e + 2] = __float_as_uint(__uint_as_float(x[e + 2]) * (rs * k4.z));
                            x[e + 3] = __float_as_uint(__uint_as_float(x[e + 3]) * (rs * k4.w));
                        }
                    }
                    const float f = is_open ? 1.f : rs;
                    if (p.cap > kWideCap) {
                        const float c2 = p.cap * kLog2eT, ic = 2.f / p.cap;
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            x[e] = __float_as_uint(capped_wide(__uint_as_float(x[e]) * f, c2, ic));
                    } else if (p.cap > 0.f) {
                        // (raw scores, with the row's factor in the exponent's; kept finite: 0 times it is 0)
                        const float c2 = p.cap * kLog2eT, fc = fminf(f * (2.f / p.cap), 3e38f);
#pragma unroll
                        for (int e = 0; e < 32; ++e) x[e] = __float_as_uint(capped(__uint_as_float(x[e]), c2, fc));
                    } else if (!is_open && !p.alibi) {
#pragma unroll
                        for (int e = 0; e < 32; ++e) x[e] = __float_as_uint(__uint_as_float(x[e]) * f);
                    }
                    const float g = p.cap > 0.f ? 1.f : f;
                    if (is_open) {
                        // visibility words of the chunk's two blocks; bit u: place u of the block
                        uint32_t vis[2];
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const int j0 = base + 32 * (2 * (c >> 1) + k) - pad;
                            uint32_t d = (1u << open) - 1u;           // the open group: seen
                            if (j0 >= 0) {
                                if (mrow) d = (j0 >> 5) < p.mask_words ? mrow[j0 >> 5] : 0u;
                                else d = t - j0 >= 31 ? 0xFFFFFFFFu : (t < j0 ? 0u : (2u << (t - j0)) - 1u);
                                if (nk - j0 < 32) d &= nk <= j0 ? 0u : (1u << (nk - j0)) - 1u;
                            }
                            vis[k] = d >> (4 * (c & 1));
                        }
                        const int4 *kp = reinterpret_cast<const int4 *>(smem + SM::kpos) + ((i & 3) * kTile + 32 * c) / 4;
                        const bool posn = p.alibi || p.window;
                        const int far = p.window ? p.window : 0x7FFFFFFF;
#pragma unroll
                        for (int e = 0; e < 32; ++e) {
                            bool see = (vis[(e >> 3) & 1] >> (tile_token(e) & 31)) & 1u;
                            if (posn) {
                                const int4 k4 = kp[e / 4];
                                const int dist = pos - ((e & 3) == 0 ? k4.x : (e & 3) == 1 ? k4.y : (e & 3) == 2 ? k4.z : k4.w);
                                x[e] = __float_as_uint(fmaf(-slope2, static_cast<float>(dist), __uint_as_float(x[e])));
                                see = see && dist < far;
                            }
                            if (!see) x[e] = 0xFF800000u;
                        }
                    } else {
                        const int o = 64 * (c >> 1) + 4 * (c & 1);   // tile_token(32 c + e) = o + tile_token(e)
                        if (p.alibi) {
                            const float d0 = -slope2 * static_cast<float>(pos - base - o);
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                x[e] = __float_as_uint(fmaf(__uint_as_float(x[e]), g,
                                                            fmaf(slope2, static_cast<float>(tile_token(e)), d0)));
                        }
                        if (cut) {
                            const uint32_t len = static_cast<uint32_t>(max(hi - lo, 0));
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                if (static_cast<uint32_t>(o + tile_token(e) - lo) >= len) x[e] = 0xFF800000u;
                        }
                    }
                };
                auto top = [&](const uint32_t *x, float mx) {
                    float a = mx, d = -INFINITY;
#pragma unroll
                    for (int e = 0; e < 32; e += 4) {
                        a = max3(a, __uint_as_float(x[e]), __uint_as_float(x[e + 1]));
                        d = max3(d, __uint_as_float(x[e + 2]), __uint_as_float(x[e + 3]));
                    }
                    return fmaxf(a, d);
                };
                const int c0 = copy * NC;                 // the row's chunks [c0, c0 + NC)
                uint32_t x[NC][32];
                if (NC > 1 && shaped) {   // shaped scores are written back, then read like plain ones
#pragma unroll 1
                    for (int c = c0; c < c0 + NC; ++c) {
                        ld32_issue(ts + 32 * c, x[0]);
                        ld32_wait(x[0]);
                        shape(x[0], c);
                        st32(ts + 32 * c, x[0]);
                    }
                    st_wait();
                }
                // ---- the row's maximum; its last two chunks stay in registers
                float mx = -INFINITY;
                if (NC == 4) {
                    ld32_issue(ts, x[0]);
                    ld32_issue(ts + 32, x[1]);
                    ld32_wait(x[0]);
                    ld32_wait(x[1]);
                    mx = top(x[1], top(x[0], mx));
                }
                constexpr int H = NC > 2 ? 2 : 0;         // first chunk that stays
#pragma unroll
                for (int c = H; c < NC; ++c) ld32_issue(ts + 32 * (c0 + c), x[c]);
#pragma unroll
                for (int c = H; c < NC; ++c) ld32_wait(x[c]);
                if (NC == 1 && shaped) shape(x[0], c0);
#pragma unroll
                for (int c = H; c < NC; ++c) mx = top(x[c], mx);
                const float f = shaped ? 1.f : rs;
                // the maximum (in log2 units) moves only when it grew by more than the lag, then O and l
                // are rescaled; O also from the open tiles' unit to the packed ones' (never smaller)
                mx *= f;
                int shift = 0;   // at the slot's first packed tile
                if (ti >= 0 && ti < step && use > 0) shift = open_exp() - ev;
                if (__any_sync(0xffffffffu, mx > m + kLag) || shift != 0) {
                    const float mn = fmaxf(m, mx);
                    if (use > 0) {
                        const float al = m == -INFINITY ? 0.f : fast_exp2(m - mn);
                        l *= al;
                        const float ao = al * pow2f(shift);
#pragma unroll 1
                        for (int c = 0; c < D / 16; ++c) {
                            uint32_t y[16];
                            ld16_issue(to + 16 * c, y);
                            ld16_wait(y);
#pragma unroll
                            for (int e = 0; e < 16; ++e) y[e] = __float_as_uint(__uint_as_float(y[e]) * ao);
                            st16(to + 16 * c, y);
                        }
                    }
                    m = mn;
                }
                // ---- weights 2^(s - m + bias), their sum, fp16 into tensor memory over the scores
                const float sub = m == -INFINITY ? 0.f : kWeightBias - m;
                const uint64_t f2 = pack2(f, f), sub2 = pack2(sub, sub);
                uint64_t sum = pack2(0.f, 0.f);
                auto weigh = [&](const uint32_t *y, int c) {
                    uint32_t pk[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const uint64_t v = fma2(pack2(__uint_as_float(y[2 * e]), __uint_as_float(y[2 * e + 1])), f2, sub2);
                        float a, d;
                        unpack2(v, a, d);
                        a = fast_exp2(a);
                        d = fast_exp2(d);
                        sum = add2(sum, pack2(a, d));
                        pk[e] = pack_h2(a, d);
                    }
                    st16(ts + kWeightCol + 16 * c, pk);
                };
                weigh(x[H], c0 + H);
                if (NC == 4) ld32_issue(ts, x[0]);
                if (NC > 1) weigh(x[H + 1], c0 + H + 1);
                if (NC == 4) {
                    ld32_wait(x[0]);
                    ld32_issue(ts + 32, x[1]);
                    weigh(x[0], 0);
                    ld32_wait(x[1]);
                    weigh(x[1], 1);
                }
                if (REP > 1) {   // the other copies' columns
                    uint32_t zero[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) zero[e] = 0u;
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        if (c / NC != copy) st16(ts + kWeightCol + 16 * c, zero);
                }
                float s0, s1;
                unpack2(sum, s0, s1);
                l += s0 + s1;
                st_wait();
            }
            fence_before();
            __syncwarp();
            arrive_one(on, &bar->p_full[j]);
        }
        // ---- the end: join slots and copies, write rows
        if (n > 0) wait(&bar->o_full[0], 0);
        if (TWO ? n > 0 : n > 1) wait(&bar->o_full[1], 0);
        fence_after();
        const bool any = first < n, final_ = p.S == 1;
        const int slots = min(n, 2);                             // slots with a tile (one row tile)
        float2 *mlx = reinterpret_cast<float2 *>(smem + SM::ml);
        float *rows_o = reinterpret_cast<float *>(smem);
        float own = 1.f;
        if (!TWO) {
            mlx[tid] = make_float2(m, l);
            asm volatile("bar.sync 1, 256;" ::: "memory");
            float M = -INFINITY;
            for (int s = 0; s < slots; ++s)
#pragma unroll
                for (int k = 0; k < REP; ++k) M = fmaxf(M, mlx[s * 128 + k * COPY + r].x);
            // (a part without a visible key has l = 0 and O = 0)
            own = m == -INFINITY ? 1.f : fast_exp2(m - M);
            l = 0.f;
            for (int s = 0; s < slots; ++s)
#pragma unroll
                for (int k = 0; k < REP; ++k) {
                    const float2 y = mlx[s * 128 + k * COPY + r];
                    l += y.x == -INFINITY ? y.y : y.y * fast_exp2(y.x - M);
                }
            m = M;
        }
        if (busy && any) {
            own *= final_ ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
            // O's unit: the slot's last tile's (a product of its own: own times it may leave fp32's range)
            const int last = TWO || ((n ^ j) & 1) ? n - 1 : n - 2;
            const float ounit = pow2f(tb + last < n_open ? open_exp() : ev);
            float *dst = rows_o + tid * SM::ROW;
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
                uint32_t x[32];
                ld32_issue(to + 32 * c, x);
                ld32_wait(x);
#pragma unroll
                for (int e = 0; e < 32; e += 4)
                    *reinterpret_cast<float4 *>(dst + 32 * c + e) =
                        make_float4(__uint_as_float(x[e]) * own * ounit, __uint_as_float(x[e + 1]) * own * ounit,
                                    __uint_as_float(x[e + 2]) * own * ounit, __uint_as_float(x[e + 3]) * own * ounit);
            }
        }
        if (!final_ && r < nrow && copy == 0 && (TWO || j == 0))
            *reinterpret_cast<float2 *>(p.part_ml + (((static_cast<long long>(b) * p.T + t) * Hq + hq) * p.sstride + sp) * 2) =
                make_float2(m, l);
        asm volatile("bar.sync 1, 256;" ::: "memory");
        const bool fix = bar->bad_value != 0;
        for (int it = tid; it < nrow * NL; it += 256) {
            const int rr = it / NL, c = 8 * (it % NL);
            const int tt = row_t(rr), hh = h * p.G + (row0 + rr) - tt * p.G;
            float o[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = 0.f;
            auto add = [&](int src) {
                const float4 x = *reinterpret_cast<const float4 *>(rows_o + src * SM::ROW + c);
                const float4 y = *reinterpret_cast<const float4 *>(rows_o + src * SM::ROW + c + 4);
                o[0] += x.x; o[1] += x.y; o[2] += x.z; o[3] += x.w;
                o[4] += y.x; o[5] += y.y; o[6] += y.z; o[7] += y.w;
            };
            if (TWO) {
                if (n > 0) add(rr);
            } else {
                for (int s = 0; s < slots; ++s)
#pragma unroll
                    for (int k = 0; k < REP; ++k) add(s * 128 + k * COPY + rr);
            }
            if (fix) {
                // NaN and infinite drafted values of this split's open tiles, where the row sees them
                const uint32_t *mr = p.mask ? p.mask + (static_cast<long long>(b) * p.T + tt) * p.mask_words : nullptr;
                const int qp = query_pos(rr);
                const int ja = max(0, kTile * tb - pad), je = min(nk, kTile * min(te, n_open) - pad);
                for (int jd = ja; jd < je; ++jd) {
                    bool see = mr ? (mr[jd >> 5] >> (jd & 31)) & 1u : jd <= tt;
                    if (p.window && qp - (L + (depth ? depth[jd] : jd)) >= p.window) see = false;
                    if (!see) continue;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float v = quant::bf16_to_f32(p.vd[(unit * p.T + jd) * D + c + e]);
                        if (!(fabsf(v) < INFINITY)) o[e] += v;
                    }
                }
            }
            const long long row = (static_cast<long long>(b) * p.T + tt) * Hq + hh;
            if (!final_ || p.out_fp32) {
                float *dst = final_ ? static_cast<float *>(p.out) + row * D + c
                                    : p.part_acc + (row * p.sstride + sp) * D + c;
                reinterpret_cast<float4 *>(dst)[0] = make_float4(o[0], o[1], o[2], o[3]);
                reinterpret_cast<float4 *>(dst)[1] = make_float4(o[4], o[5], o[6], o[7]);
            } else {
                uint32_t w4[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const __nv_bfloat162 v = __floats2bfloat162_rn(o[2 * k], o[2 * k + 1]);
                    w4[k] = *reinterpret_cast<const uint32_t *>(&v);
                }
                *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.out) + row * D + c) = make_uint4(w4[0], w4[1], w4[2], w4[3]);
            }
        }
    }
    if (wait.failed) atomicOr(p.status, kStatusWaitExpired);
    fence_before();
    __syncthreads();
    if (warp == 16)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols));
}

// Joins the splits of every live row: a warp per row, partials in log2 units.
template <int D>
__global__ void __launch_bounds__(256) tree_merge_kernel(const TreeParams p) {
    pdl_enter();
    const int Hq = p.Hkv * p.G, lane = threadIdx.x & 31;
    const long long row = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    if (row >= static_cast<long long>(p.B) * p.T * Hq) return;
    const int b = static_cast<int>(row / Hq / p.T), t = static_cast<int>(row / Hq % p.T);
    if (t >= p.len.queries(b)) return;
    const float2 *ml = reinterpret_cast<const float2 *>(p.part_ml) + row * p.sstride;
    float M = -INFINITY;
    for (int s = 0; s < p.S; ++s) M = fmaxf(M, ml[s].x);
    constexpr int PER = D / 32;
    // NaN and infinities that a row sees are added at full weight, as in a launch without splits: a
    // weight of zero must not meet them
    float o[PER], bad[PER], den = 0.f;
#pragma unroll
    for (int e = 0; e < PER; ++e) o[e] = bad[e] = 0.f;
    for (int s = 0; s < p.S; ++s) {
        const float2 v = ml[s];
        const float w = v.x == -INFINITY ? 0.f : fast_exp2(v.x - M);   // 0: a split without a visible key
        den += v.x == -INFINITY ? v.y : w * v.y;
        const float *a = p.part_acc + (row * p.sstride + s) * D + PER * lane;
#pragma unroll
        for (int e = 0; e < PER; ++e) {
            const bool fin = fabsf(a[e]) < INFINITY;
            o[e] = fmaf(w, fin ? a[e] : 0.f, o[e]);
            bad[e] += fin ? 0.f : a[e];
        }
    }
    const float n = den == 0.f ? 0.f : 1.f / den;
#pragma unroll
    for (int e = 0; e < PER; e += 2) {
        const float x = fmaf(o[e], n, bad[e]), y = fmaf(o[e + 1], n, bad[e + 1]);
        const long long at = row * D + PER * lane + e;
        if (p.out_fp32) *reinterpret_cast<float2 *>(static_cast<float *>(p.out) + at) = make_float2(x, y);
        else *reinterpret_cast<__nv_bfloat162 *>(static_cast<__nv_bfloat16 *>(p.out) + at) = __floats2bfloat162_rn(x, y);
    }
}

constexpr int kSmemMax = 232448;

int part_bytes(int D, int bits) { return 4 * D * bits + 4 * D; }
int fixed_bytes(int D, bool two) {
    if (D == 128) return two ? TreeSmem<128, true>::ring : TreeSmem<128, false>::ring;
    return two ? TreeSmem<64, true>::ring : TreeSmem<64, false>::ring;
}
static_assert(TreeSmem<128, true>::ring + 8 * (4 * 128 * 8 + 4 * 128) <= kSmemMax, "one stage of every part fits");

std::mutex g_tree_mu;
bool g_tree_set[64][8];   // per device ordinal: shared-memory limits raised

}  // namespace

int tree_row_groups(int rows) { return (rows + 255) / 256; }

// Partials are sized for at most four CTAs per SM.
int tree_max_splits(int B, int Hkv, int rows) {
    const long long ctas = static_cast<long long>(B) * Hkv * tree_row_groups(rows);
    return static_cast<int>(std::max(1LL, std::min(64LL, 4LL * kSms / ctas)));
}

int tree_splits(int B, int Hkv, int row_groups, long long tiles, int max_splits) {
    const long long ctas = static_cast<long long>(B) * Hkv * row_groups;
    double best = 1e300;
    int S = 1;
    for (int s = 1; s <= max_splits && s <= tiles; ++s) {
        const double waves = static_cast<double>((ctas * s + kSms - 1) / kSms);
        const double cost = waves * (static_cast<double>((tiles + s - 1) / s) + 4.0) + (s > 1 ? 2.0 : 0.0);
        if (cost < best - 1e-9) {
            best = cost;
            S = s;
        }
    }
    return S;
}

cudaError_t launch_tree(const TreeParams &p0, int D, cudaStream_t st) {
    TreeParams p = p0;
    const int rows = p.T * p.G;
    const bool two = rows > kTile;
    const int groups = tree_row_groups(rows);
    // stages of the packed parts: as many as fit, up to four, the fewer-staged kind first
    const int pk = part_bytes(D, p.bk), pv = part_bytes(D, p.bv), fixed = fixed_bytes(D, two);
    p.dk = p.dv = 1;
    for (bool more = true; more;) {
        more = false;
        int *x = p.dk <= p.dv ? &p.dk : &p.dv;
        for (int k = 0; k < 2 && !more; ++k, x = x == &p.dk ? &p.dv : &p.dk) {
            if (*x >= 4) continue;
            ++*x;
            if (fixed + 4 * (p.dk * pk + p.dv * pv) <= kSmemMax) more = true;
            else --*x;
        }
    }
    const int smem = std::max(fixed + 4 * (p.dk * pk + p.dv * pv), 120 * 1024);   // one CTA per SM (its 512 TMEM columns)
    using Fn = void (*)(const TreeParams);
    // copies: as many as the rows leave room for (four: each softmax warp takes 32 of a tile's
    // 128 columns instead of one warp taking them all)
    const int rep = two || rows > 64 ? 1 : (rows > 32 ? 2 : 4);
    const Fn fn = D == 128 ? (two ? tree_kernel<128, true, 1> : rep == 1 ? tree_kernel<128, false, 1>
                              : rep == 2 ? tree_kernel<128, false, 2> : tree_kernel<128, false, 4>)
                           : (two ? tree_kernel<64, true, 1> : rep == 1 ? tree_kernel<64, false, 1>
                              : rep == 2 ? tree_kernel<64, false, 2> : tree_kernel<64, false, 4>);
    {
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        std::lock_guard<std::mutex> lk(g_tree_mu);
        const int slot = (D == 128 ? 4 : 0) + (two ? 3 : rep >> 1);
        if (dev >= 64 || !g_tree_set[dev][slot]) {
            e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax);
            if (e != cudaSuccess) return e;
            if (dev < 64) g_tree_set[dev][slot] = true;
        }
    }
    cudaError_t e = launch_pdl(fn, dim3(p.S, p.Hkv * groups, p.B), dim3(kTreeThreads), smem, st, p);
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_tree_merge(const TreeParams &p, int D, cudaStream_t st) {
    const long long rows = static_cast<long long>(p.B) * p.T * p.Hkv * p.G;
    const dim3 grid(static_cast<unsigned>((rows + 7) / 8));
    cudaError_t e = D == 128 ? launch_pdl(tree_merge_kernel<128>, grid, dim3(256), 0, st, p)
                             : launch_pdl(tree_merge_kernel<64>, grid, dim3(256), 0, st, p);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace kvq
