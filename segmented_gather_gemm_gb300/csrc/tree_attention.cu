// Attention of draft trees over the paged cache (include/csgmv.h,
// csgmv_tree_attention).
//
// Mathematics.  For the rows of one request and kv head (its drafted tokens
// times the query heads of the group, cut into tiles of 128) and tiles of 128
// tokens: S = Q K^T, a running maximum m and sum l of the softmax in base 2,
// O <- 2^(m - m') O + P V with P = 2^(scale log2(e) S - m').  m' moves only
// when it would grow by more than 2^8 (P stays below 2^8, so fp32 sums lose
// nothing), which keeps O in tensor memory untouched on almost every tile.
//
// What bounds it.  A tile of K and V (64 KB at head_dim 128) takes an SM's
// share of HBM 1.47 us; its two products at 128 rows take the tensor core
// 0.7 us and the exponentials of 128 x 128 scores 0.6 us.  So bytes bound it up
// to about 128 rows for each kv head.
//
// Few rows.  Up to 16 rows (plain decoding) the products are turned over: S^T =
// K Q^T and O^T = V^T P^T with the tokens (the elements of V) down the 128
// lanes and 16 columns of rows, P^T in shared memory.  The tensor core then does
// an eighth of the work, and that counts although it has time for all of it:
// with 128-row products the power limit lowers the clock (1.3 to 1.6 GHz).
//
// More rows.  The exponentials of a full tile take an SM 512 clocks, all of the
// softmax's instructions some 800; what costs is the latency of its steps (read
// S, find the maximum, exponentials, store P).  A warp has 16 rows: four threads
// share a row, and no warp waits for another.  (Sixteen warps of 32 rows by 32
// tokens, agreeing on a row's maximum through shared memory, stayed in step
// with one another: 1950 clocks a tile in half, 2250 in bfloat16, against 1570
// and 1770.)
//
// Split.  The tiles of all (request, kv head, row tile) items form one axis
// that is cut into parts of equal cost (cost_of below), one a CTA (one CTA an
// SM), so a batch of ragged lengths and a single long sequence both fill the
// GPU.  An item cut by the ends of a part leaves fp32 partial sums in the
// workspace (at most two a CTA), which a second kernel joins in order of the
// axis: results do not depend on timing.
//
// More than 128 rows.  Taken one after the other, the row tiles of a head each
// read its K and V from HBM: a head's tokens do not stay in L2 while an SM goes
// through them.  So two CTAs may share a part and walk it together, each with
// one of two row tiles, the second to ask for a tile of K and V finding it in
// L2.  That doubles a part's length, and the CTA whose row tile is missing or
// small waits; every CTA adds up the cost of both ways and takes the cheaper
// (`ways`).  32 trees of 33 to 64 tokens, 4 query heads a kv head, 500 to 8192
// cached: 145 us together, 199 us apart.  (Both row tiles in one CTA, K and V
// read once, took 221 us when this took 174: each tile then waits for the
// other's softmax, products and their hand-overs.)
//
// Rounding.  Half inputs round P to half, scaled by 2^4 so that small weights
// keep their bits; bfloat16 would keep 8 bits, as coarse as the output's own
// rounding, so there P goes in as a high part (its upper 16 bits) and what that
// leaves, rounded, in two products, which the tensor core has time for.  Half
// weights have 11 bits, as the output has; turned over their low part costs
// nothing and goes in as well, above 16 rows it would cost a quarter: the trees
// below 192 us instead of 152 (called one by one), for a largest error of
// 8.3e-4, the output's rounding alone, instead of 1.07e-3.
//
// One CTA: a warp each fills a ring of K tiles and one of V tiles with TMA, a
// warp issues S = Q K^T up to three tiles ahead (three S buffers, each P in its
// S's place), a warp issues O += P V, eight warps do the softmax from tensor
// memory.  An MMA takes 75 to 100 clocks to issue here, whatever its size, and a
// wait that is over 150; one warp for both products was busy 2330 clocks a tile
// and held everything up (bfloat16, head_dim 64, 128 rows a kv head over 100003
// and 131072 tokens: 73 us, with two warps 63.5 us).
//
// Waits are bounded.  After one has run out nothing of the call's results holds,
// but its warps meet at all barriers and wait for their own copies and products;
// calls that find the status bit do nothing (what this takes: trees 145 to 147 us).
//
// Measured now: that case 58 to 60 us; 256 requests of one token, 64 to 4096
// cached, 8 kv heads of 128, 328 us (6.7 TB/s, 98 % of a plain copy's rate); a
// tree of 12 over 1021 tokens 12.6 us.

#include <cudaTypedefs.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <atomic>

#include "serving.cuh"

namespace csgmv {
namespace {

constexpr int kTile = 128;         // rows of a row tile, tokens of a token tile
constexpr int kGroups = kTile / 8; // 8-row groups: the unit of the shared-memory layout
constexpr int kAttnCtas = 152;     // one CTA an SM
constexpr int kSoftWarps = 8;
constexpr int kWarpK = kSoftWarps, kWarpV = kWarpK + 1, kWarpS = kWarpK + 2, kWarpO = kWarpK + 3;
constexpr int kAttnThreads = 32 * (kSoftWarps + 4);
constexpr int kBufs = 3;           // S buffers in tensor memory, P^T buffers in shared memory
constexpr int kWalks = 4;          // items that the product warp has told the others of
constexpr int kMaxRequests = 16000;  // 12 bytes each in the tiles' memory
constexpr int kCombineThreads = 128;
constexpr float kLazy = 8.0f;      // growth of the maximum (base 2) that is let stand
constexpr float kLog2e = 1.4426950408889634f;

template <int D>
struct Shape {
    static constexpr int kHalves = D / 64;             // 128-byte column blocks of a row
    static constexpr int kGroupBytes = kHalves * 1024; // 8 rows
    static constexpr int kTileBytes = kGroups * kGroupBytes;
    static constexpr int kSlotsK = D == 128 ? 2 : 5, kSlotsV = D == 128 ? 3 : 5;  // of the rings
    static constexpr int kRings = (kSlotsK + kSlotsV) * kTileBytes;
    static constexpr int kBars = 2 * (kSlotsK + kSlotsV) + 3 * kBufs + 1 + 2 * kWalks + 2;
    static constexpr int kQBytes = 32768;               // Q of an item, or 16 rows of it and P^T
    static constexpr int kTiles = 2 * kQBytes + kRings;  // Q of two items, and the rings
    static_assert(kTileBytes <= kQBytes && 8192 + kBufs * 8192 <= kQBytes, "Q and P^T");
    static constexpr int kRedBytes = 3 * kTile * 4;     // a row's maximum and sum; the same turned over, by warps
    static constexpr int kFlagBytes = 2 * 8 * 4;       // a warp's flag, by turns
    static constexpr int kWalkBytes = kWalks * 32;
    static constexpr int kBarsAt = kTiles + kRedBytes + kFlagBytes + kWalkBytes;
    static constexpr int kSmem = kBarsAt + (kBars + 1) * 8 + 64;
    static_assert((kTiles + kRedBytes + kFlagBytes) % 16 == 0 && kBarsAt % 8 == 0, "alignment");
    static_assert(kTile == 128, "items() shifts by 7");
    static_assert(kSmem <= 227 * 1024, "shared memory");
    static_assert(512 + 12 * kMaxRequests + 32 <= kTiles, "what the axis is cut by");
};

struct AttnMaps {
    CUtensorMap k, v;    // whole boxes of a page
    CUtensorMap k8, v8;  // 8 rows of a page
    CUtensorMap kn, vn;  // 8 rows of the drafted tokens
};
enum { kPagesGeneral = 0, kPagesHeadsOut = 1, kPagesHeadsIn = 2 };

struct Parts {  // of the items that the cuts go through
    float *part;      // [2 * kAttnCtas][D / 4][kTile] float4: unscaled O
    float *ml;        // [2 * kAttnCtas][2][kTile]: m, l
    int4 *starters;   // [kAttnCtas]: the item a CTA begins and does not end {first token, h, first row, rows and ways}, or {-1}
    int *tails;       // [kAttnCtas]: of an item begun by an earlier CTA: 0 nothing, 1 a middle part, 2 its end
};
struct AttnKernelParams : Parts {
    AttnParams p;
    AttnMaps maps;
    int form;         // kPages*
    int box_groups;   // 8-row groups of a whole box
};

__device__ __forceinline__ void tma_load_5d(uint32_t dst, const void *tmap, int c0, int c1, int c2, int c3, int c4,
                                            uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, "
        "%6}], [%7];\n" ::"r"(dst),
        "l"(tmap), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4), "r"(smem_u32(bar))
        : "memory");
}

// Shared-memory matrix descriptor, 128-byte (or 64-byte) swizzle: `lbo` the
// distance of whole swizzle widths along the contiguous dimension (used when
// that is not K), `sbo` the distance of 8-row groups.
__device__ __forceinline__ uint64_t smem_desc(uint32_t saddr, uint32_t lbo, uint32_t sbo, bool swizzle64 = false) {
    return (uint64_t)((saddr >> 4) & 0x3FFF) | (uint64_t)((lbo >> 4) & 0x3FFF) << 16 |
           (uint64_t)((sbo >> 4) & 0x3FFF) << 32 | (uint64_t)1 << 46 | (uint64_t)(swizzle64 ? 4 : 2) << 61;
}
// Instruction descriptor of kind::f16, fp32 accumulation; `a_mn` / `b_mn`: A /
// B is stored with its M / N dimension contiguous.
__device__ __forceinline__ uint32_t idesc16(bool f16, int M, int N, bool a_mn, bool b_mn) {
    const uint32_t fmt = f16 ? 0u : 1u;
    return (1u << 4) | fmt << 7 | fmt << 10 | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u) |
           (uint32_t)(N >> 3) << 17 | (uint32_t)(M >> 4) << 24;
}
// MMAs and commits that every lane of a warp reaches and the one with `lead`
// issues: the warp's control flow stays uniform, so descriptors live in
// uniform registers and an MMA costs few issue slots, which it shares with
// the softmax warps of its scheduler.
__device__ __forceinline__ void mma_ss(uint32_t lead, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
        " @q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add), "r"(lead)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t lead, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
        " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)add), "r"(lead)
        : "memory");
}
__device__ __forceinline__ void commit_one(uint32_t lead, uint64_t *bar) {
    asm volatile(
        "{\n .reg .pred q;\n setp.ne.b32 q, %1, 0;\n"
        " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(smem_u32(bar)),
        "r"(lead)
        : "memory");
}
__device__ __forceinline__ uint32_t elect_lead() {
    uint32_t r;
    asm volatile("{\n .reg .pred q;\n elect.sync _|q, 0xffffffff;\n selp.u32 %0, 1, 0, q;\n}\n" : "=r"(r));
    return r;
}
// Two fp32 numbers in one 64-bit register: one instruction for two of the same
// operation (as long as two, but half the issue slots).
__device__ __forceinline__ uint64_t two(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};\n" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 apart(uint64_t x) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;\n" : "=f"(r.x), "=f"(r.y) : "l"(x));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;\n" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
    return y;
}
// Tensor memory, 8 columns of 32 lanes: a thread has a lane.
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, float (&v)[8]) {
    uint32_t r[8];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {"
        "%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n"
        "tcgen05.wait::ld.sync.aligned;\n"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
        : "r"(taddr)
        : "memory");
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&v)[8]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {"
        "%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
        : "memory");
}
// 16 lanes, 8 columns a step i: thread z has columns 8 i + 2 (z & 3) and the one
// after of lanes z / 4 (v[4 i], v[4 i + 1]) and 8 + z / 4 (v[4 i + 2], v[4 i + 3]).
__device__ __forceinline__ void tmem_ld_rows128(uint32_t taddr, float (&v)[64]) {
    uint32_t r[64];
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x16.b32 {"
        "%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,"
        "%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,"
        "%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%64];\n"
        "tcgen05.wait::ld.sync.aligned;\n"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]), "=r"(r[32]),
          "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]), "=r"(r[40]),
          "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]), "=r"(r[48]),
          "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]), "=r"(r[56]),
          "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
        : "r"(taddr)
        : "memory");
#pragma unroll
    for (int i = 0; i < 64; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_ld_rows64(uint32_t taddr, float (&v)[32]) {
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x8.b32 {"
        "%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
        "tcgen05.wait::ld.sync.aligned;\n"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_st_rows64(uint32_t taddr, const uint32_t (&v)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.16x256b.x8.b32 [%0], {"
        "%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};\n" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]),
        "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]),
        "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
        : "memory");
}
// 16 lanes, 4 columns a step i: column 4 i + (z & 3) of the same two lanes.
__device__ __forceinline__ void tmem_st_rows64x1(uint32_t taddr, const uint32_t (&v)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.16x128b.x16.b32 [%0], {"
        "%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};\n" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]),
        "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]),
        "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
        : "memory");
}

template <bool F16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    if (F16) {
        const __half2 v = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&v);
    }
    return pack_bf16x2(lo, hi);
}
// What packing two numbers to 16 bits left of them, packed.
template <bool F16>
__device__ __forceinline__ uint32_t pack2_rest(uint32_t packed, float lo, float hi) {
    float2 h;
    if (F16) h = __half22float2(*reinterpret_cast<const __half2 *>(&packed));
    else h = unpack_bf16x2(packed);
    return pack2<F16>(lo - h.x, hi - h.y);
}
template <bool F16>
__device__ __forceinline__ bool nonfinite16(uint32_t x) {
    const uint32_t e = F16 ? 0x7c00u : 0x7f80u;
    return (x & e) == e;
}
template <bool F16>
__device__ __forceinline__ float widen(uint16_t x) {
    return F16 ? __half2float(__ushort_as_half(x)) : __uint_as_float((uint32_t)x << 16);
}

// One request's part of the work.  Tokens lie on a virtual axis: the cached
// ones, padded to whole 8-row groups, then the drafted ones.
struct Req {
    int lo, T, L, slot;
    __device__ __forceinline__ int ctx_groups() const { return (L + 7) >> 3; }
    __device__ __forceinline__ int groups() const { return ctx_groups() + ((T + 7) >> 3); }
    __device__ __forceinline__ int token_tiles() const { return (groups() + kGroups - 1) / kGroups; }
    __device__ __forceinline__ int items(int group, int ways) const { return (T * group + kTile * ways - 1) >> (6 + ways); }  // ways is 1 or 2
};

// Request b, with T = 0 (no work) when it is not sound; the status bit why.
__device__ __forceinline__ Req load_req(const AttnParams &p, int b, int *bad) {
    Req r;
    r.lo = p.indptr[b];
    const int hi = p.indptr[b + 1];
    r.slot = p.slots ? p.slots[b] : b;
    r.T = hi - r.lo;
    r.L = 0;
    *bad = 0;
    if (r.lo < 0 || hi < r.lo || hi > p.num_tokens || (p.mask && r.T > 32 * p.mask_words)) *bad = CSGMV_KV_STATUS_BAD_LENS;
    else if (r.slot < 0 || r.slot >= p.max_seqs) *bad = CSGMV_KV_STATUS_BAD_SEQ;
    else {
        r.L = p.seq_lens[r.slot];
        if (r.L < 0 || r.L > p.max_pages * p.page_size) *bad = CSGMV_KV_STATUS_BAD_LENS;
    }
    if (*bad) r.T = r.L = 0;
    return r;
}

constexpr int kFewRows = 16;  // up to so many rows the products are turned over

// What the parts of the axis are weighed by, in units of 64 clocks.  Measured
// on long axes: a tile's K and V of head_dim 128 come in 2870 clocks of an SM's
// share of HBM, half of that when two CTAs read them together (of head_dim 64 in
// 1430); its softmax takes 1000 clocks turned over, otherwise 1400 (half) or 1700
// (bfloat16).  (Bytes of head_dim 64 are weighed as the turned-over softmax, which
// is too little where that is all there is: no such batch has been measured.)  Beginning and ending an item costs
// 5800 turned over (its tiles' loads start anew), 10200 otherwise.  With equal
// tile counts instead, 256 requests of 64 to 4096 tokens take 340 us (328), the
// trees above 218 us (145).
//
// An item's cost fits 29 bits (2^30 tokens); a head's, and the batch's, may pass
// 32: those are 64 bits wide, and the axis counts in steps of 2^shift units where
// 31 bits of them would not do (`scale_of`).
struct Cost {
    int mi, nt;          // items and token tiles
    int tile[2], item[2];  // of a full item, of the last: one token tile, the whole item
    long long head;      // a kv head's items
};
// More than so many units (2^40: four minutes of the whole GPU) are refused.
constexpr long long kMaxCost = 1ll << 40;
__device__ __forceinline__ int scale_of(long long all, int bs) {
    int shift = 0;
    while ((all >> shift) + bs > INT32_MAX) ++shift;  // (a request's share is rounded up)
    return shift;
}
__device__ __forceinline__ int tile_cost(int rows, bool shared, int d, bool f16) {
    const int bytes = (d == 128 ? 45 : 16) >> (int)shared;
    return max(bytes, rows <= kFewRows ? 16 : f16 ? 22 : 26);
}
__device__ __forceinline__ int item_cost(int rows) { return rows <= kFewRows ? 90 : 160; }
__device__ __forceinline__ Cost cost_of(int T, int L, const AttnParams &p, int ways) {
    Cost c;
    const Req r = {0, T, L, 0};
    c.mi = r.items(p.group, ways);
    c.nt = r.token_tiles();
    const int rest = T * p.group - (c.mi - 1) * ways * kTile, last = min(kTile, rest);  // the last item's rows, its first tile's
    c.tile[0] = tile_cost(kTile, ways == 2, p.d, p.f16);
    c.tile[1] = tile_cost(last, rest > kTile, p.d, p.f16);
    c.item[0] = item_cost(kTile) + c.nt * c.tile[0];
    c.item[1] = item_cost(last) + c.nt * c.tile[1];
    c.head = (long long)(c.mi - 1) * c.item[0] + c.item[1];
    return c;
}
// A request's cost, no more than one past what is refused (so that sums of 16000 stay in range).
__device__ __forceinline__ long long request_cost(int T, int L, const AttnParams &p, int ways) {
    return T ? min(cost_of(T, L, p, ways).head * p.hkv, kMaxCost + 1) : 0;
}

// A place on the axis: token tile t of an item.
struct Place {
    int b, h, m, t;
    __device__ __forceinline__ bool same_item(int b2, int h2, int m2) const { return b == b2 && h == h2 && m == m2; }
};

// A CTA's part of the axis, walked item by item.
struct Walk {
    Req r;
    int b, h, m, t0;   // request, kv head, row tile, first token tile of the segment
    int n, nt;         // token tiles of the segment, of the item
    Place end;         // first tile past the part
    __device__ __forceinline__ bool cut() {
        n = (end.same_item(b, h, m) ? min(end.t, nt) : nt) - t0;
        return n > 0;
    }
    // (`ways` row tiles are an item, of which the CTA has one.)
    __device__ __forceinline__ bool next(const AttnParams &p, int ways) {
        do {
            if (end.same_item(b, h, m)) return false;
            t0 = 0;
            const int way = blockIdx.x & (ways - 1);
            m += ways;
            if ((m - way) * kTile >= r.T * p.group) {
                m = way;
                if (++h == p.hkv) {
                    h = 0;
                    do {
                        if (++b >= p.bs) return false;
                        int bad;
                        r = load_req(p, b, &bad);
                    } while (r.T == 0 && b < end.b);
                    if (r.T == 0) return false;
                    nt = r.token_tiles();
                }
            }
            if (!cut()) return false;
        } while (rows(p) <= 0);  // an item without this way's row tile
        return true;
    }
    __device__ __forceinline__ int rows(const AttnParams &p) const { return min(kTile, r.T * p.group - m * kTile); }
};

// 32 bits of row t's mask from drafted token j0 (which may be negative: lower
// bits are then 0), cut at T.
__device__ __forceinline__ uint32_t tree_word(const AttnParams &p, const Req &r, int t, int j0) {
    uint32_t x;
    const int a = max(j0, 0), w = a >> 5;
    if (p.mask) {
        const int32_t *row = p.mask + (int64_t)(r.lo + t) * p.mask_words;
        const uint32_t w0 = w < p.mask_words ? (uint32_t)row[w] : 0u, w1 = w + 1 < p.mask_words ? (uint32_t)row[w + 1] : 0u;
        x = __funnelshift_r(w0, w1, a & 31);
    } else {
        const int n = t + 1 - a;
        x = n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u;
    }
    if (j0 < 0) x = j0 > -32 ? x << -j0 : 0u;
    const int lim = r.T - j0;
    return lim >= 32 ? x : lim <= 0 ? 0u : x & ((1u << lim) - 1u);
}

// The place x steps of 2^shift units of cost along the axis (every CTA rounds
// it alike).  `ahead`: steps before each request, and the total; `tl`: their T
// and L.
__device__ __forceinline__ Place place_at(const AttnParams &p, const int *ahead, const int2 *tl, int ways, int shift, int x) {
    Place q = {p.bs, 0, 0, 0};
    if (x >= ahead[p.bs]) return q;
    int lo = 0, hi = p.bs;  // the last request with ahead <= x: it has work of its own
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (ahead[mid] <= x) lo = mid; else hi = mid;
    }
    const Cost c = cost_of(tl[lo].x, tl[lo].y, p, ways);
    q.b = lo;
    // (without a shift everything fits 32 bits, and the divisions are short)
    const long long in_request = (long long)(x - ahead[lo]) << shift;
    q.h = shift ? (int)(in_request / c.head) : (int)in_request / (int)c.head;
    const long long in_head = in_request - q.h * c.head;
    q.m = min(shift ? (int)(in_head / c.item[0]) : (int)in_head / c.item[0], c.mi - 1);
    int y = (int)(in_head - (long long)q.m * c.item[0]);
    const int last = q.m == c.mi - 1, cost = c.tile[last];
    y -= c.item[last] - c.nt * cost;
    q.t = y <= 0 ? 0 : (y + cost - 1) / cost;
    if (q.t >= c.nt) {  // the next item's beginning
        q.t = 0;
        if (++q.m == c.mi) {
            q.m = 0;
            if (++q.h == p.hkv) {
                q.h = 0;
                do ++q.b; while (q.b < p.bs && ahead[q.b + 1] == ahead[q.b]);
            }
        }
    }
    return q;
}

// What row t sees of the non-finite values of the drafted tokens in n token
// tiles from t0 on, at element el of V: they are added in the end.
template <bool F16>
__device__ __noinline__ float odd_sum(const AttnParams &p, Req r, int h, int t, int el, int t0, int n) {
    float sum = 0.0f;
    for (int j = max(0, t0 * kTile - r.ctx_groups() * 8); j < min(r.T, (t0 + n) * kTile - r.ctx_groups() * 8); ++j) {
        const uint16_t v = p.v_new[(int64_t)(r.lo + j) * p.n_ts + h * p.n_hs + el];
        if (nonfinite16<F16>(v) && (tree_word(p, r, t, j) & 1)) sum += widen<F16>(v);
    }
    return sum;
}

// Q of an item into its swizzled tile, by `threads` threads (a multiple of
// D / 8) of which this is thread `i`: each has one 16-byte column.
template <int D>
__device__ __forceinline__ void fetch_q(const AttnParams &p, const Walk &w, unsigned char *q_s, int i, int threads) {
    const int rows = w.rows(p), chunk = i % (D / 8), step = threads / (D / 8);
    int row = i / (D / 8), t = (w.m * kTile + row) / p.group, g = w.m * kTile + row - t * p.group;
    const uint16_t *src = p.q + (int64_t)(w.r.lo + t) * p.q_ts + (w.h * p.group + g) * p.q_hs + chunk * 8;
    for (; row < rows; row += step) {
        cp_async16(q_s + (row >> 3) * Shape<D>::kGroupBytes + (row & 7) * 128 + (chunk >> 3) * 1024 + (((chunk & 7) ^ (row & 7)) << 4),
                   src, 16);
        g += step;
        src += step * p.q_hs;
        while (g >= p.group) {  // the next token
            g -= p.group;
            src += p.q_ts - p.group * p.q_hs;
        }
    }
}
__device__ __forceinline__ void q_landed() {
    asm volatile("cp.async.wait_all;\n" ::: "memory");
    fence_proxy_async_smem();
}

template <int D, bool F16>
__global__ void __launch_bounds__(kAttnThreads, 1) attend(const __grid_constant__ AttnKernelParams k) {
    using S = Shape<D>;
    const AttnParams &p = k.p;
    extern __shared__ __align__(1024) unsigned char smem[];
    unsigned char *q_s = smem, *k_ring = q_s + 2 * S::kQBytes, *v_ring = k_ring + S::kSlotsK * S::kTileBytes;
    float *red_s = reinterpret_cast<float *>(smem + S::kTiles);
    int *flag_s = reinterpret_cast<int *>(smem + S::kTiles + S::kRedBytes);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + S::kBarsAt);
    uint64_t *k_full = bars, *k_empty = k_full + S::kSlotsK, *v_full = k_empty + S::kSlotsK, *v_empty = v_full + S::kSlotsV,
             *s_full = v_empty + S::kSlotsV, *p_ready = s_full + kBufs, *pv_done = p_ready + kBufs,
             *q_ready = pv_done + kBufs, *walk_full = q_ready + 1, *walk_empty = walk_full + kWalks,
             *drained = walk_empty + kWalks;
    uint32_t *misc = reinterpret_cast<uint32_t *>(bars + S::kBars + 1);
    int4 *walk_s = reinterpret_cast<int4 *>(smem + S::kTiles + S::kRedBytes + S::kFlagBytes);
    // The last item with a non-finite drafted V, of the even and of the odd ones: a softmax warp may be in the
    // next item while another still ends this one (not two on, for a product takes P of all of them).
    volatile int *odd_item = reinterpret_cast<volatile int *>(misc + 4);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

    // (The join is not launched early: its blocks among this kernel's cost 12 us a call.)
    if (smem_u32(smem) & 1023) {  // the swizzled tiles count on it
        if (tid == 0) {
            atomicOr(p.status, CSGMV_KV_STATUS_TIMEOUT);
            k.starters[blockIdx.x] = make_int4(-1, 0, 0, 0);
        }
        return;
    }
    if (warp == kWarpO) {
        tmem_alloc(misc, 512);
        tmem_relinquish();
    }
    if (tid == 0) {
        for (int i = 0; i < 2 * (S::kSlotsK + S::kSlotsV); ++i) mbar_init(&bars[i], 1);
        for (int i = 0; i < kBufs; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_ready[i], kSoftWarps);
            mbar_init(&pv_done[i], 1);
        }
        mbar_init(q_ready, kSoftWarps);
        for (int i = 0; i < kWalks; ++i) {
            mbar_init(&walk_full[i], 1);
            mbar_init(&walk_empty[i], kSoftWarps + 1);
        }
        for (int i = 0; i < 2; ++i) mbar_init(&drained[i], 1);
        fence_mbar_init();
        odd_item[0] = odd_item[1] = -1;
    }
    griddep_wait();
    // A wait that ran out in an earlier call (or in this one, elsewhere): waits would no longer be sat out.
    const bool stuck = tid == 0 && (*reinterpret_cast<volatile int32_t *>(p.status) & CSGMV_KV_STATUS_TIMEOUT) != 0;
    // The axis: cost ahead of each request, and its T and L, in the tiles' memory.
    int *ahead = reinterpret_cast<int *>(smem + 512);
    int2 *tl = reinterpret_cast<int2 *>(smem + 512 + ((4 * p.bs + 4 + 15) & ~15));
    Place *ends = reinterpret_cast<Place *>(smem);
    long long all = 0;
    int ways = 1, shift = 0, lo = 0, slot = 0;  // (the last two of request `tid`)
    {
        long long *ws = reinterpret_cast<long long *>(smem + 64);
        long long shared = 0, tot;  // of two CTAs that walk together
        for (int b0 = 0; b0 < p.bs; b0 += kAttnThreads) {
            const int b = b0 + tid;
            long long n = 0;
            if (b < p.bs) {
                int bad;
                const Req r = load_req(p, b, &bad);
                n = request_cost(r.T, r.L, p, 1);
                shared += request_cost(r.T, r.L, p, 2);
                tl[b] = make_int2(r.T, r.L);
                if (b0 == 0) lo = r.lo, slot = r.slot;
                if (bad && blockIdx.x == 0) atomicOr(p.status, bad);
            }
            const long long pre = block_scan_ex(n, ws, &tot);
            if (b < p.bs) ahead[b] = (int)min(all + pre, (long long)INT32_MAX);  // counted again below where that cuts it
            all += tot;
        }
        if (p.num_tokens * p.group > kTile && gridDim.x > 1) {
            block_scan_ex(shared, ws, &tot);
            if (2 * tot < all) ways = 2, all = tot;
        }
        if (all > kMaxCost) {  // refused
            if (blockIdx.x == 0 && tid == 0) atomicOr(p.status, CSGMV_KV_STATUS_CAPACITY);
            all = 0;
        } else if (ways == 2 || all > INT32_MAX) {
            shift = scale_of(all, p.bs);
            all = 0;
            for (int b0 = 0; b0 < p.bs; b0 += kAttnThreads) {
                const int b = b0 + tid;
                const long long n = b < p.bs ? (request_cost(tl[b].x, tl[b].y, p, ways) + (1ll << shift) - 1) >> shift : 0;
                const long long pre = block_scan_ex(n, ws, &tot);
                if (b < p.bs) ahead[b] = (int)(all + pre);
                all += tot;
            }
        }
    }
    if (__syncthreads_or(stuck)) all = 0;
    if (tid == 0) ahead[p.bs] = (int)all;
    __syncthreads();
    // this CTA's part: two warps find its two ends
    if (lane == 0 && warp < 2) {
        const int parts = gridDim.x >> (ways - 1), q = (int)all / parts, rest = (int)all - q * parts,
                  c = (blockIdx.x >> (ways - 1)) + warp;
        ends[warp] = place_at(p, ahead, tl, ways, shift, c < parts ? c * q + min(c, rest) : (int)all);
    }
    if (tid == 0) {
        k.starters[blockIdx.x] = make_int4(-1, 0, 0, 0);
        k.tails[blockIdx.x] = 0;
    }
    __syncthreads();
    // its first request: known to a thread, if there is one for each
    const bool known = p.bs <= kAttnThreads;
    if (known && tid == ends[0].b) walk_s[0] = make_int4(lo, tl[tid].x, tl[tid].y, slot);
    __syncthreads();
    Walk w0 = {};
    {
        const Place at = ends[0];
        const int way = blockIdx.x & (ways - 1);
        w0.b = at.b;
        w0.h = at.h;
        w0.m = at.m * ways + way;
        w0.t0 = at.t;
        w0.end = ends[1];
        w0.end.m = w0.end.m * ways + way;
    }
    bool idle = all == 0 || w0.b >= p.bs;
    if (!idle) {
        int bad;
        const int4 r = walk_s[0];
        w0.r = known ? Req{r.x, r.y, r.z, r.w} : load_req(p, w0.b, &bad);
        w0.nt = w0.r.token_tiles();
        idle = !w0.cut() || (w0.rows(p) <= 0 && !w0.next(p, ways));
    }
    fence_proxy_async_smem();  // the tiles' memory goes over to TMA
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = misc[0];
    const uint32_t t_o = tmem + kBufs * 128;

    // After a wait that ran out (status bit TIMEOUT, results meaningless) every warp still comes to the same
    // items and meets every barrier that others wait at.  But a warp whose loads have no place to go stops
    // them (also when the place is free by the barriers' count and what it held has not landed), and the
    // warps of loads and products wait in the end for what they have in flight: nothing may write to shared
    // or tensor memory that the CTA has given back.
    constexpr uint64_t kDrain = 2000000000ull;
    auto within = [&](uint64_t *bar, uint32_t parity, uint64_t ns) {  // a bounded wait that does not look at the status
        if (mbar_try_wait(bar, parity)) return true;
        const uint64_t t0 = global_ns();
        do {
            if (mbar_try_wait(bar, parity)) return true;
        } while (global_ns() - t0 < ns);
        atomicOr(p.status, CSGMV_KV_STATUS_TIMEOUT);
        return false;
    };

    // The next item, from the warp that multiplies Q and K to those that do the rest (none: n = 0), in
    // one of kWalks places, written again only when every one of them has read it.  Neither wait can last,
    // for all others are bounded and both sides come here in turn.
    constexpr uint64_t kLong = 20000000000ull;
    auto tell = [&](const Walk &w, int item) {
        const int at = (item - 1) % kWalks, round = (item - 1) / kWalks;
        if (lane == 0) {
            if (round > 0) within(&walk_empty[at], (round - 1) & 1, kLong);
            walk_s[2 * at] = make_int4(w.r.lo, w.r.T, w.r.L, w.h);
            walk_s[2 * at + 1] = make_int4(w.m, w.t0, w.n, w.nt);
            mbar_arrive(&walk_full[at]);
        }
    };
    auto told = [&](Walk &w, int item) {
        const int at = (item - 1) % kWalks, phase = ((item - 1) / kWalks) & 1;
        if (!__all_sync(kFullMask, within(&walk_full[at], phase, kLong))) return false;
        __syncwarp();
        const int4 a = walk_s[2 * at], b = walk_s[2 * at + 1];
        __syncwarp();
        if (lane == 0) mbar_arrive(&walk_empty[at]);
        w.r.lo = a.x;
        w.r.T = a.y;
        w.r.L = a.z;
        w.h = a.w;
        w.m = b.x;
        w.t0 = b.y;
        w.n = b.z;
        w.nt = b.w;
        return w.n > 0;
    };

    if (idle) {
        // nothing
    } else if (warp == kWarpK || warp == kWarpV) {
        // ------------------------------------------------------------ loads
        const bool v = warp == kWarpV;
        const void *map_page = v ? &k.maps.v : &k.maps.k, *map_8 = v ? &k.maps.v8 : &k.maps.k8,
                   *map_new = v ? &k.maps.vn : &k.maps.kn;
        uint64_t *full = v ? v_full : k_full, *empty = v ? v_empty : k_empty;
        const uint32_t ring = smem_u32(v ? v_ring : k_ring);
        if (lane == 0) {
            prefetch_tmap(map_page);
            prefetch_tmap(map_8);
            prefetch_tmap(map_new);
        }
        const int gpp_shift = __ffs(p.page_size >> 3) - 1;  // log2 of the 8-row groups of a page
        const int bg = k.box_groups;
        // the page a lane's load of token tile t needs (0 where it needs none)
        auto page_of = [&](const Walk &w, int t) {
            const int g = t * kGroups + lane, whole = (w.r.L >> 3) & ~(bg - 1);
            const bool ctx = lane < kGroups && g < w.r.ctx_groups();
            return ctx && (g >= whole || !(lane & (bg - 1))) ? p.page_table[(int64_t)w.r.slot * p.max_pages + (g >> gpp_shift)] : 0;
        };
        const int slots = v ? S::kSlotsV : S::kSlotsK;
        int s = 0, phase = 0;  // of the ring
        Walk w = w0, wn = w0;
        int page = page_of(w, w.t0);
        bool more, on = true;
        do {
            more = wn.next(p, ways);  // looked up while this segment's tiles are loaded
            const int gctx = w.r.ctx_groups(), gall = w.r.groups();
            const int whole = (w.r.L >> 3) & ~(bg - 1);  // groups in boxes that are full of tokens
            for (int t = w.t0; t < w.t0 + w.n; ++t) {
                const int next_page = t + 1 < w.t0 + w.n ? page_of(w, t + 1) : more ? page_of(wn, wn.t0) : 0;
                const int g = t * kGroups + lane, ng = min(kGroups, gall - t * kGroups);
                const bool in = lane < ng, ctx = in && g < gctx;
                const bool box = ctx && g < whole, lead = box && !(lane & (bg - 1));
                if (page < 0 || page >= p.num_pages) {
                    atomicOr(p.status, CSGMV_KV_STATUS_BAD_PAGE);
                    page = p.num_pages;  // past the pool: zeros
                }
                const int rg = g & ((1 << gpp_shift) - 1);
                on = mbar_wait(&empty[s], phase ^ 1, p.status, CSGMV_KV_STATUS_TIMEOUT);
                on &= mbar_try_wait(&full[s], phase ^ 1);  // (so it is, but for waits that ran out)
                if (!(on = __all_sync(kFullMask, on))) break;
                if (lane == 0) mbar_arrive_expect_tx(&full[s], (uint32_t)ng * S::kGroupBytes);
                __syncwarp();
                const uint32_t dst = ring + s * S::kTileBytes + lane * S::kGroupBytes;
                if (lead) {
                    if (k.form == kPagesHeadsOut) tma_load_5d(dst, map_page, 0, 0, 0, rg, page * p.hkv + w.h, &full[s]);
                    else if (k.form == kPagesHeadsIn) tma_load_5d(dst, map_page, 0, 0, 0, w.h, (page << gpp_shift) + rg, &full[s]);
                    else tma_load_5d(dst, map_page, 0, rg * 8, 0, w.h, page, &full[s]);
                } else if (ctx && !box) {
                    tma_load_5d(dst, map_8, 0, rg * 8, 0, w.h, page, &full[s]);
                } else if (in && !ctx) {
                    tma_load_5d(dst, map_new, 0, w.r.lo + (g - gctx) * 8, 0, w.h, 0, &full[s]);
                }
                page = next_page;
                if (++s == slots) s = 0, phase ^= 1;
            }
            w = wn;
        } while (more && on);
        // each place's last load (from the place before s on back, once around the ring)
        for (int i = 0; i < slots; ++i) within(&full[i], i < s ? phase : phase ^ 1, kDrain);
    } else if (warp == kWarpS) {
        // ------------------------------------------------ products: S = Q K^T
        const uint32_t lead = elect_lead();
        const uint32_t id_few = idesc16(F16, kTile, 16, false, false);
        const uint64_t q_d = smem_desc(smem_u32(q_s), 16, S::kGroupBytes), k_d = smem_desc(smem_u32(k_ring), 16, S::kGroupBytes);
        int it = 0, item = 0;
        Walk w = w0;
        bool more;
        do {
            Walk wn = w;
            more = wn.next(p, ways);
            const int gall = w.r.groups();
            const bool few = w.rows(p) <= kFewRows;
            if (item == 0) mbar_wait(q_ready, 0, p.status, CSGMV_KV_STATUS_TIMEOUT);  // the softmax warps fetch the first
            else q_landed();
            __syncwarp();
            for (int t = w.t0; t < w.t0 + w.n; ++t, ++it) {
                const int s = it % S::kSlotsK, buf = it % kBufs;
                // what the buffer held has been read, and P that lay in its place multiplied
                if (it >= kBufs) mbar_wait(&pv_done[buf], ((it / kBufs) & 1) ^ 1, p.status, CSGMV_KV_STATUS_TIMEOUT);
                mbar_wait(&k_full[s], (it / S::kSlotsK) & 1, p.status, CSGMV_KV_STATUS_TIMEOUT);
                __syncwarp();
                tc_fence_after();
                const int steps = (min(kGroups, gall - t * kGroups) + 1) >> 1;  // of 16 tokens
                const uint32_t id = idesc16(F16, kTile, 16 * steps, false, false), dst = tmem + buf * 128;
                const uint64_t kd = k_d + (uint32_t)(s * S::kTileBytes >> 4), qd = q_d + (uint32_t)((item & 1) * S::kQBytes >> 4);
                if (few) {
#pragma unroll
                    for (int x = 0; x < D / 16; ++x) {
                        const uint32_t off = ((x / 4) * 1024 + (x % 4) * 32) >> 4;
                        mma_ss(lead, dst, kd + off, qd + off, id_few, x > 0);
                    }
                } else {
#pragma unroll
                    for (int x = 0; x < D / 16; ++x) {
                        const uint32_t off = ((x / 4) * 1024 + (x % 4) * 32) >> 4;
                        mma_ss(lead, dst, qd + off, kd + off, id, x > 0);
                    }
                }
                commit_one(lead, &k_empty[s]);
                commit_one(lead, &s_full[buf]);
                if (more && t == w.t0 + min(2, w.n - 1)) {
                    // Q of the next item, where Q and P^T of the one before were: its last product is done
                    const int last = it - (t - w.t0) - 1;
                    if (last >= 0) mbar_wait(&pv_done[last % kBufs], (last / kBufs) & 1, p.status, CSGMV_KV_STATUS_TIMEOUT);
                    fetch_q<D>(p, wn, q_s + ((item + 1) & 1) * S::kQBytes, lane, 32);
                }
            }
            ++item;
            w = wn;
            if (!more) w.n = 0;
            tell(w, item);
        } while (more);
        commit_one(lead, &drained[0]);
        within(&drained[0], 0, kDrain);
    } else if (warp == kWarpO) {
        // ------------------------------------------------ products: O += P V
        const uint32_t lead = elect_lead();
        const uint32_t id_pv = idesc16(F16, kTile, D, false, true), id_few = idesc16(F16, kTile, 32, true, true);
        const uint64_t v_d = smem_desc(smem_u32(v_ring), 1024, S::kGroupBytes), p_d = smem_desc(smem_u32(q_s) + 8192, 16, 512, true);
        int it = 0, item = 0;
        Walk w = w0;
        do {
            const int gall = w.r.groups();
            const bool few = w.rows(p) <= kFewRows;
            for (int t = w.t0; t < w.t0 + w.n; ++t, ++it) {
                const int s = it % S::kSlotsV, buf = it % kBufs;
                mbar_wait(&v_full[s], (it / S::kSlotsV) & 1, p.status, CSGMV_KV_STATUS_TIMEOUT);
                mbar_wait(&p_ready[buf], (it / kBufs) & 1, p.status, CSGMV_KV_STATUS_TIMEOUT);
                __syncwarp();
                tc_fence_after();
                const int steps = (min(kGroups, gall - t * kGroups) + 1) >> 1;  // of 16 tokens
                const uint64_t vd = v_d + (uint32_t)(s * S::kTileBytes >> 4), pd = p_d + (uint32_t)(((item & 1) * S::kQBytes + buf * 8192) >> 4);
                const uint32_t pt = tmem + buf * 128;
                const bool add = t > w.t0;
                if (few) {
#pragma unroll
                    for (int x = 0; x < 8; ++x)
                        if (x < steps)
                            mma_ss(lead, t_o, vd + (uint32_t)(x * 2 * S::kGroupBytes >> 4), pd + (uint32_t)(x * 1024 >> 4),
                                   id_few, add || x > 0);
                } else {
#pragma unroll
                    for (int x = 0; x < 8; ++x) {
                        if (x < steps) {
                            // P lies in 64 columns, its low parts in the next 64
                            const uint64_t d = vd + (uint32_t)(x * 2 * S::kGroupBytes >> 4);
                            mma_ts(lead, t_o, pt + 8 * x, d, id_pv, add || x > 0);
                            if (!F16) mma_ts(lead, t_o, pt + 64 + 8 * x, d, id_pv, true);
                        }
                    }
                }
                commit_one(lead, &v_empty[s]);
                commit_one(lead, &pv_done[buf]);
            }
        } while (told(w, ++item));
        commit_one(lead, &drained[1]);
        within(&drained[1], 0, kDrain);
    } else {
        // ---------------------------------------------------------- softmax
        // warps w and w + 4 share 32 lanes (a quadrant)
        const int quad = warp & 3, half = warp >> 2, pos = quad * 32 + lane;
        const uint32_t lane_base = (uint32_t)(quad * 32) << 16;
        const float c = p.scale * kLog2e;
        constexpr float kShift = F16 ? 4.0f : 0.0f;  // P up to 2^12 in half: small weights keep more of their bits
        int it = 0, item = 0;
        Walk w = w0;

        fetch_q<D>(p, w, q_s, tid, kSoftWarps * 32);
        q_landed();
        __syncwarp();
        if (lane == 0) mbar_arrive(q_ready);

        do {
            const int rows = w.rows(p);
            const bool few = rows <= kFewRows;
            const int gctx = w.r.ctx_groups(), gall = w.r.groups();
            const bool whole = w.n == w.nt;
            const int cell = 2 * (int)blockIdx.x + (w.t0 == 0 ? 1 : 0);
            auto keys_of = [&](int t) { return ((min(kGroups, gall - t * kGroups) + 1) >> 1) * 16; };
            auto edge = [&](int t) { return (t + 1) * kTile > w.r.L; };  // holds more than cached tokens
            auto await_s = [&]() {
                mbar_wait(&s_full[it % kBufs], (it / kBufs) & 1, p.status, CSGMV_KV_STATUS_TIMEOUT);
                __syncwarp();
                tc_fence_after();
            };
            // (A warp may get here before another has P of the tile before last ready: the barrier is
            // the buffer's own, so the parity cannot be that of an older product.)
            auto await_pv = [&]() {  // of the tile before
                mbar_wait(&pv_done[(it - 1) % kBufs], ((it - 1) / kBufs) & 1, p.status, CSGMV_KV_STATUS_TIMEOUT);
                __syncwarp();
                tc_fence_after();
            };
            // V of an edge tile.  Rows that are no token are cleared (a weight of 0 would not silence a
            // NaN there); what is not finite in a drafted row is taken out, and added at the end to the
            // rows that see it.
            auto clean_v = [&](int t) {
                const int sv = it % S::kSlotsV;
                mbar_wait(&v_full[sv], (it / S::kSlotsV) & 1, p.status, CSGMV_KV_STATUS_TIMEOUT);
                const int r0 = max(w.r.L - t * kTile, 0), n = (keys_of(t) - r0) * (D / 8);
                for (int i = tid; i < n; i += kSoftWarps * 32) {
                    const int r = r0 + i / (D / 8), y = i % (D / 8), jt = t * kTile + r - gctx * 8;
                    uint4 *a = reinterpret_cast<uint4 *>(v_ring + sv * S::kTileBytes + (r >> 3) * S::kGroupBytes +
                                                         (r & 7) * 128 + (y >> 3) * 1024 + (y & 7) * 16);
                    uint4 v = make_uint4(0, 0, 0, 0);
                    bool odd = true;
                    if (jt >= 0 && jt < w.r.T) {
                        v = *a;
                        uint32_t *e = reinterpret_cast<uint32_t *>(&v);
                        odd = false;
#pragma unroll
                        for (int z = 0; z < 4; ++z) {
                            if (nonfinite16<F16>(e[z])) odd = true, e[z] &= 0xffff0000u;
                            if (nonfinite16<F16>(e[z] >> 16)) odd = true, e[z] &= 0x0000ffffu;
                        }
                        if (odd) odd_item[item & 1] = item;
                    }
                    if (odd) *a = v;
                }
                fence_proxy_async_smem();
            };
            auto p_is_ready = [&]() {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_ready[it % kBufs]);
            };
            auto inverse = [](float l) { return l > 0.0f ? 1.0f / l : l == 0.0f ? 0.0f : l; };  // NaN stays
            auto put_row = [&](int row, float m, float l) {  // what a row leaves beside O
                if (!whole) {
                    k.ml[cell * 2 * kTile + row] = m;
                    k.ml[cell * 2 * kTile + kTile + row] = l;
                } else if (p.lse) {
                    const int at = w.m * kTile + row, t = at / p.group;
                    p.lse[(int64_t)(w.r.lo + t) * p.hq + w.h * p.group + (at - t * p.group)] =
                        l == 0.0f ? -INFINITY : (m + (log2f(l) - kShift)) * 0.6931471805599453f;
                }
            };

            if (few) {
                // ------------------------------------------- turned over
                // a thread has token `pos` and rows 8 half .. 8 half + 7, of which nl are real
                const int nl = min(8, rows - 8 * half);
                float m[8], l[8];
#pragma unroll
                for (int r = 0; r < 8; ++r) m[r] = -INFINITY, l[r] = 0.0f;
                for (int j = 0; j < w.n; ++j, ++it) {
                    const int t = w.t0 + j, buf = it % kBufs;
                    await_s();
                    if (nl > 0) {
                        float s[8];
                        tmem_ld8(tmem + buf * 128 + lane_base + 8 * half, s);
                        uint32_t see = (1u << nl) - 1u;
                        const int vk = t * kTile + pos;
                        if (vk >= w.r.L) {
                            const int jt = vk - gctx * 8;
                            uint32_t bits = 0;
                            if (jt >= 0 && jt < w.r.T)
                                for (int r = 0; r < nl; ++r)
                                    bits |= (tree_word(p, w.r, (w.m * kTile + 8 * half + r) / p.group, jt) & 1u) << r;
                            see &= bits;
                        }
                        __syncwarp();
                        bool grow = false;
#pragma unroll
                        for (int r = 0; r < 8; ++r) {
                            s[r] = (see >> r) & 1 ? s[r] : -INFINITY;
                            grow |= s[r] * c > m[r] + kLazy;  // from -inf: any score at all
                        }
                        // whether any of the half's four warps has a score past its maximum's leeway
                        const bool mine = __any_sync(kFullMask, grow);
                        int *flags = flag_s + (it & 1) * 8 + half * 4;
                        if (lane == 0) flags[quad] = mine;
                        named_bar_sync(5 + half, 128);
                        const int4 any = *reinterpret_cast<const int4 *>(flags);
                        if (any.x | any.y | any.z | any.w) {
                            float *mx = red_s + 2 * kTile + half * 64;  // [quadrant][row]
#pragma unroll
                            for (int r = 0; r < 8; ++r) {
                                float x = s[r] * c;
#pragma unroll
                                for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(kFullMask, x, o));
                                if (lane == 0) mx[quad * 8 + r] = x;
                            }
                            named_bar_sync(5 + half, 128);
                            float f[8];
#pragma unroll
                            for (int r = 0; r < 8; ++r) {
                                const float x = fmaxf(fmaxf(mx[r], mx[8 + r]), fmaxf(mx[16 + r], mx[24 + r]));
                                const float mn = x > m[r] + kLazy ? x : m[r];
                                f[r] = mn > m[r] ? ex2(m[r] - mn) : 1.0f;
                                m[r] = mn;
                                l[r] *= f[r];
                            }
                            if (j > 0) {  // O^T so far
                                await_pv();
#pragma unroll
                                for (int part = 0; part < 2; ++part) {
                                    const uint32_t a = t_o + lane_base + part * 16 + half * 8;
                                    float o[8];
                                    uint32_t u[8];
                                    tmem_ld8(a, o);
#pragma unroll
                                    for (int r = 0; r < 8; ++r) u[r] = __float_as_uint(o[r] * f[r]);
                                    tmem_st8(a, u);
                                }
                                tmem_wait_st();
                            }
                        }
                        uint32_t hi[4], low[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            float e[2];
#pragma unroll
                            for (int y = 0; y < 2; ++y) {
                                const int r = 2 * i + y;
                                e[y] = ex2(fmaf(s[r], c, m[r] == -INFINITY ? 0.0f : kShift - m[r]));
                                l[r] += e[y];
                            }
                            hi[i] = pack2<F16>(e[0], e[1]);
                            low[i] = pack2_rest<F16>(hi[i], e[0], e[1]);
                        }
                        if (it >= kBufs)  // the product before in this buffer
                            mbar_wait(&pv_done[buf], ((it / kBufs) & 1) ^ 1, p.status, CSGMV_KV_STATUS_TIMEOUT);
                        // P^T: 64 bytes a token, high parts of 16 rows, then the low parts; 64-byte swizzle
                        const uint32_t a = smem_u32(q_s) + (item & 1) * S::kQBytes + 8192 + buf * 8192 + pos * 64, x = (pos >> 1) & 3;
                        asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};\n" ::"r"(a + ((half ^ x) << 4)), "r"(hi[0]), "r"(hi[1]),
                                     "r"(hi[2]), "r"(hi[3])
                                     : "memory");
                        asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};\n" ::"r"(a + (((2 + half) ^ x) << 4)), "r"(low[0]),
                                     "r"(low[1]), "r"(low[2]), "r"(low[3])
                                     : "memory");
                    }
                    if (edge(t)) clean_v(t);
                    else fence_proxy_async_smem();
                    p_is_ready();
                }
                if (nl > 0) {
                    float *sum = red_s + 2 * kTile + half * 64 + 32;  // [quadrant][row], beside the maxima
#pragma unroll
                    for (int r = 0; r < 8; ++r) {
                        l[r] = warp_sum(l[r]);
                        if (lane == 0) sum[quad * 8 + r] = l[r];
                    }
                    named_bar_sync(5 + half, 128);
#pragma unroll
                    for (int r = 0; r < 8; ++r) l[r] = (sum[r] + sum[8 + r]) + (sum[16 + r] + sum[24 + r]);
                }
                await_pv();
                if (nl > 0) {
                    float o[8], low[8];
                    tmem_ld8(t_o + lane_base + half * 8, o);
                    tmem_ld8(t_o + lane_base + 16 + half * 8, low);
                    if (pos < D) {  // a thread has element `pos`
                        const bool odd = odd_item[item & 1] == item;
                        float *part = k.part + ((int64_t)cell * (D / 4) + pos / 4) * kTile * 4 + (pos & 3);
#pragma unroll
                        for (int r = 0; r < 8; ++r) {
                            if (r < nl) {
                                const int row = 8 * half + r, at = w.m * kTile + row, tr = at / p.group;
                                float x = o[r] + low[r];
                                if (odd) x += odd_sum<F16>(p, w.r, w.h, tr, pos, w.t0, w.n);
                                if (whole)
                                    p.out[(int64_t)(w.r.lo + tr) * p.o_ts + (w.h * p.group + (at - tr * p.group)) * p.o_hs + pos] =
                                        (uint16_t)pack2<F16>(x * inverse(l[r]), 0.0f);
                                else part[row * 4] = x;
                                if (pos == 0) put_row(row, m[r], l[r]);
                            }
                        }
                    }
                }
            } else {
                // ------------------------------------------------- as is
                // a warp has 16 rows, a thread two of them: elements 2 z, 2 z + 1 of every 8 tokens
                // (z its number in the four that share the rows)
                const int row0 = quad * 32 + half * 16 + lane / 4, z = lane & 3;
                const bool warp_live = quad * 32 + half * 16 < rows;
                const uint32_t lanes = (uint32_t)(quad * 32 + half * 16) << 16;
                const bool live[2] = {row0 < rows, row0 + 8 < rows};
                float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};  // base 2, m without kShift; l of this thread's tokens
                for (int j = 0; j < w.n; ++j, ++it) {
                    const int t = w.t0 + j;
                    await_s();
                    if (warp_live) {
                        const uint32_t t_s = tmem + (it % kBufs) * 128 + lanes;
                        float s[64];
                        tmem_ld_rows128(t_s, s);
                        if (edge(t)) {
                            // a thread looks up two of its rows' eight words: words z of both
                            const int k0 = t * kTile + 32 * z, n = w.r.L - k0;
                            uint32_t see[2];
#pragma unroll
                            for (int r = 0; r < 2; ++r) {
                                const int tr = min((w.m * kTile + row0 + 8 * r) / p.group, w.r.T - 1);
                                see[r] = tree_word(p, w.r, tr, k0 - gctx * 8) | (n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u);
                            }
#pragma unroll
                            for (int q = 0; q < 4; ++q) {
#pragma unroll
                                for (int r = 0; r < 2; ++r) {
                                    const uint32_t bits = __shfl_sync(kFullMask, see[r], q, 4) >> (2 * z);
#pragma unroll
                                    for (int i = 0; i < 8; ++i) {
                                        float &x = s[16 * q + 4 * (i / 2) + 2 * r + i % 2];
                                        x = (bits >> (8 * (i / 2) + i % 2)) & 1 ? x : -INFINITY;
                                    }
                                }
                            }
                        }
                        float top[2];
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            float mx[2] = {s[2 * r], s[2 * r + 1]};
#pragma unroll
                            for (int i = 1; i < 15; i += 2) {
                                mx[0] = max3(mx[0], s[4 * i + 2 * r], s[4 * i + 2 * r + 1]);
                                mx[1] = max3(mx[1], s[4 * i + 4 + 2 * r], s[4 * i + 4 + 2 * r + 1]);
                            }
                            float x = fmaxf(max3(mx[0], s[60 + 2 * r], s[60 + 2 * r + 1]), mx[1]);
                            x = fmaxf(x, __shfl_xor_sync(kFullMask, x, 1));
                            top[r] = fmaxf(x, __shfl_xor_sync(kFullMask, x, 2)) * c;
                        }
                        // from -inf: any score at all
                        const bool grow[2] = {live[0] && top[0] > m[0] + kLazy, live[1] && top[1] > m[1] + kLazy};
                        if (__any_sync(kFullMask, grow[0] || grow[1])) {
                            float f[2];
#pragma unroll
                            for (int r = 0; r < 2; ++r) {
                                f[r] = grow[r] ? ex2(m[r] - top[r]) : 1.0f;  // m = -inf: 0
                                m[r] = grow[r] ? top[r] : m[r];
                                l[r] *= f[r];
                            }
                            if (j > 0) {  // O so far, in units of 2^m
                                await_pv();
#pragma unroll
                                for (int h = 0; h < D / 64; ++h) {
                                    float o[32];
                                    uint32_t u[32];
                                    tmem_ld_rows64(t_o + lanes + 64 * h, o);
#pragma unroll
                                    for (int i = 0; i < 32; ++i) u[i] = __float_as_uint(o[i] * f[(i / 2) & 1]);
                                    tmem_st_rows64(t_o + lanes + 64 * h, u);
                                }
                            }
                        }
                        const uint64_t c2 = two(c, c), minus = two(-1.0f, -1.0f);
                        uint64_t base2[2], sum[2] = {0, 0};
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            const float base = m[r] == -INFINITY ? 0.0f : kShift - m[r];
                            base2[r] = two(base, base);
                        }
                        uint32_t u[32], low[32];
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            const float2 x = apart(fma2(two(s[2 * i], s[2 * i + 1]), c2, base2[i & 1]));
                            const float e0 = ex2(x.x), e1 = ex2(x.y);
                            const uint64_t e = two(e0, e1);
                            sum[i & 1] = add2(sum[i & 1], e);
                            if (F16) {
                                u[i] = pack2<F16>(e0, e1);
                            } else {
                                const uint32_t b0 = __float_as_uint(e0), b1 = __float_as_uint(e1);
                                u[i] = __byte_perm(b0, b1, 0x7632);
                                const uint64_t high = two(__uint_as_float(b0 & 0xffff0000u), __uint_as_float(b1 & 0xffff0000u));
                                const float2 r = apart(fma2(high, minus, e));
                                low[i] = pack2<F16>(r.x, r.y);
                            }
                        }
                        tmem_st_rows64x1(t_s, u);
                        if (!F16) tmem_st_rows64x1(t_s + 64, low);
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            const float2 both = apart(sum[r]);
                            l[r] += both.x + both.y;
                        }
                        tmem_wait_st();
                    }
                    if (edge(t)) clean_v(t);
                    p_is_ready();
                }
                // From here a thread has a row, and half of O's columns.  (All warps have ended the item
                // before when the last product of this one is done: red_s can be written.)
                await_pv();
                if (quad * 32 < rows) {
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        l[r] += __shfl_xor_sync(kFullMask, l[r], 1);
                        l[r] += __shfl_xor_sync(kFullMask, l[r], 2);
                        if (z == 0) {
                            red_s[row0 + 8 * r] = m[r];
                            red_s[kTile + row0 + 8 * r] = l[r];
                        }
                    }
                    named_bar_sync(1 + quad, 64);
                    const bool odd = odd_item[item & 1] == item;
                    const float mr = red_s[pos], lr = red_s[kTile + pos], inv = inverse(lr);
                    const int at = w.m * kTile + pos, t_row = at / p.group, head = w.h * p.group + (at - t_row * p.group);
#pragma unroll 1
                    for (int h = 0; h < D / 64; ++h) {
                        const int el = half * (D / 2) + 32 * h;
                        uint16_t *dst = p.out + (int64_t)(w.r.lo + t_row) * p.o_ts + head * p.o_hs + el;
                        float *part = k.part + (((int64_t)cell * (D / 4) + el / 4) * kTile + pos) * 4;
                        float o[32];
                        tmem_ld32(t_o + lane_base + el, o);
                        if (pos < rows) {
                            if (whole) {
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    uint4 v;
                                    v.x = pack2<F16>(o[8 * i] * inv, o[8 * i + 1] * inv);
                                    v.y = pack2<F16>(o[8 * i + 2] * inv, o[8 * i + 3] * inv);
                                    v.z = pack2<F16>(o[8 * i + 4] * inv, o[8 * i + 5] * inv);
                                    v.w = pack2<F16>(o[8 * i + 6] * inv, o[8 * i + 7] * inv);
                                    *reinterpret_cast<uint4 *>(dst + i * 8) = v;
                                }
                            } else {
#pragma unroll
                                for (int i = 0; i < 8; ++i)
                                    *reinterpret_cast<float4 *>(part + i * kTile * 4) =
                                        make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                            }
                            if (odd) {
#pragma unroll 1
                                for (int i = 0; i < 32; ++i) {
                                    const float x = odd_sum<F16>(p, w.r, w.h, t_row, el + i, w.t0, w.n);
                                    if (x == 0.0f) continue;
                                    if (whole) dst[i] = (uint16_t)pack2<F16>(x * inv, 0.0f);
                                    else part[(i / 4) * kTile * 4 + (i & 3)] = x;
                                }
                            }
                        }
                        __syncwarp();
                    }
                    if (pos < rows && half == 0) put_row(pos, mr, lr);
                }
            }
            if (tid == 0 && !whole) {
                if (w.t0 == 0) k.starters[blockIdx.x] = make_int4(w.r.lo, w.h, w.m * kTile, rows | ways << 16);
                else k.tails[blockIdx.x] = w.t0 + w.n == w.nt ? 2 : 1;
            }
            tc_fence_before();
        } while (told(w, ++item));
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    __syncwarp();
    if (warp == kWarpO) tmem_dealloc(tmem, 512);
}

// What joining them takes of AttnParams.
struct JoinParams {
    uint16_t *out;
    float *lse;
    int64_t o_ts, o_hs;
    int hq, group;
};

// Joins the parts of the items that the axis' cuts went through, in order of
// the axis.  The rows of all such items are dealt out to the blocks R at a
// time.  Two rounds of dependent loads: which items and parts there are, and
// the parts (O and its scales together).
template <int D, bool F16>
__global__ void __launch_bounds__(kCombineThreads) combine(const Parts k, const JoinParams p, int ctas) {
    constexpr int R = kCombineThreads / (D / 4);  // rows of a block
    static_assert(2 * kCombineThreads >= kAttnCtas, "two items a thread");
    __shared__ int first[2 * kCombineThreads + 1], ws[33], tails[2 * kCombineThreads];
    __shared__ int4 items[2 * kCombineThreads];
    const int tid = threadIdx.x;
    griddep_launch_dependents();
    griddep_wait();
    int mine[2], all;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int c = 2 * tid + i;
        items[c] = c < ctas ? k.starters[c] : make_int4(-1, 0, 0, 0);
        tails[c] = c < ctas ? k.tails[c] : 0;
        mine[i] = items[c].x < 0 ? 0 : ((items[c].w & 0xffff) + R - 1) / R;
    }
    const int pre = block_scan_ex(mine[0] + mine[1], ws, &all);
    first[2 * tid] = pre;
    first[2 * tid + 1] = pre + mine[0];
    if (tid == 0) first[2 * kCombineThreads] = all;
    __syncthreads();
    for (int job = blockIdx.x; job < all; job += gridDim.x) {
        int c0 = 0;  // the last CTA with first <= job: it begins an item
        for (int hi = 2 * kCombineThreads; hi - c0 > 1;) {
            const int mid = (c0 + hi) >> 1;
            if (first[mid] <= job) c0 = mid; else hi = mid;
        }
        const int4 head4 = items[c0];
        const int r = tid / (D / 4), d4 = tid % (D / 4), row = (job - first[c0]) * R + r;
        const int ways = head4.w >> 16;
        if (row < (head4.w & 0xffff)) {
            // the CTAs with a part of it: up to the first that holds its end.  Sums in base 2^m of
            // the largest maximum so far
            float m = -INFINITY, l = 0.0f;
            float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            constexpr int U = 8;  // parts in flight
            bool end = false;
            for (int c = c0; c < ctas && !end; c += U * ways) {
                float ms[U], ls[U];
                float4 v[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int cu = c + u * ways, cell = 2 * cu + (cu == c0 ? 1 : 0);
                    const bool has = !end && cu < ctas && (cu == c0 || tails[cu] != 0);
                    ms[u] = -INFINITY;
                    ls[u] = 0.0f;
                    v[u] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    if (has) {
                        ms[u] = k.ml[cell * 2 * kTile + row];
                        ls[u] = k.ml[cell * 2 * kTile + kTile + row];
                        v[u] = reinterpret_cast<const float4 *>(k.part)[((int64_t)cell * (D / 4) + d4) * kTile + row];
                        end = cu != c0 && tails[cu] == 2;
                    }
                }
                float top = m;
#pragma unroll
                for (int u = 0; u < U; ++u) top = fmaxf(top, ms[u]);
                const float base = top == -INFINITY ? 0.0f : top, f = ex2(m - base);
                l *= f;
                o.x *= f;
                o.y *= f;
                o.z *= f;
                o.w *= f;
                m = top;
#pragma unroll
                for (int u = 0; u < U; ++u) {  // (a part of nothing but masked tokens has m = -inf and O = 0)
                    const float g = ex2(ms[u] - base);
                    l += ls[u] * g;
                    o.x += v[u].x * g;
                    o.y += v[u].y * g;
                    o.z += v[u].z * g;
                    o.w += v[u].w * g;
                }
            }
            constexpr float kShift = F16 ? 4.0f : 0.0f;
            const int at = head4.z + row, t = at / p.group, head = head4.y * p.group + (at - t * p.group);
            const float inv = l > 0.0f ? 1.0f / l : l == 0.0f ? 0.0f : l;
            uint2 u;
            u.x = pack2<F16>(o.x * inv, o.y * inv);
            u.y = pack2<F16>(o.z * inv, o.w * inv);
            *reinterpret_cast<uint2 *>(p.out + (int64_t)(head4.x + t) * p.o_ts + head * p.o_hs + d4 * 4) = u;
            if (d4 == 0 && p.lse)
                p.lse[(int64_t)(head4.x + t) * p.hq + head] =
                    l == 0.0f ? -INFINITY : (m + (log2f(l) - kShift)) * 0.6931471805599453f;
        }
    }
}

// ---------------------------------------------------------------- host side
std::atomic<PFN_cuTensorMapEncodeTiled_v12000> g_encode{nullptr};
constexpr int kMaxDevices = 64;
std::atomic<int> g_ready[kMaxDevices];  // CTAs to launch; 0: not set up yet (twice does no harm)

cudaError_t prepare(int *ctas) {
    int dev;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < kMaxDevices && (*ctas = g_ready[dev].load(std::memory_order_acquire)) != 0) return cudaSuccess;
    if (!g_encode) {
        void *fn = nullptr;
        cudaDriverEntryPointQueryResult q;
        e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q);
        if (e != cudaSuccess) return e;
        if (q != cudaDriverEntryPointSuccess || !fn) return cudaErrorNotSupported;
        g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
    }
    int sms = 0;
    if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
    const struct { const void *fn; int smem; } all[] = {
        {reinterpret_cast<const void *>(attend<64, false>), Shape<64>::kSmem},
        {reinterpret_cast<const void *>(attend<64, true>), Shape<64>::kSmem},
        {reinterpret_cast<const void *>(attend<128, false>), Shape<128>::kSmem},
        {reinterpret_cast<const void *>(attend<128, true>), Shape<128>::kSmem},
        {reinterpret_cast<const void *>(combine<64, false>), 0},
        {reinterpret_cast<const void *>(combine<64, true>), 0},
        {reinterpret_cast<const void *>(combine<128, false>), 0},
        {reinterpret_cast<const void *>(combine<128, true>), 0}};
    for (const auto &f : all) {
        if (f.smem && (e = cudaFuncSetAttribute(f.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, f.smem)) != cudaSuccess)
            return e;
        // both kernels with the same split of L1: an SM drains to change it
        if ((e = cudaFuncSetAttribute(f.fn, cudaFuncAttributePreferredSharedMemoryCarveout,
                                      cudaSharedmemCarveoutMaxShared)) != cudaSuccess)
            return e;
    }
    *ctas = sms < kAttnCtas ? sms : kAttnCtas;
    if (dev < kMaxDevices) g_ready[dev].store(*ctas, std::memory_order_release);
    return cudaSuccess;
}

// A 5-D map of 16-bit elements with 128-byte rows: dims and box from the
// innermost, strides in elements of dims 1 .. 4.
bool encode(CUtensorMap *map, const void *base, bool f16, const int64_t (&dim)[5], const int64_t (&stride)[4],
            const int (&box)[5]) {
    cuuint64_t d[5], s[4];
    cuuint32_t b[5], es[5] = {1, 1, 1, 1, 1};
    for (int i = 0; i < 5; ++i) {
        d[i] = (cuuint64_t)dim[i];
        b[i] = (cuuint32_t)box[i];
    }
    // the stride of a dimension of one element is never used
    for (int i = 0; i < 4; ++i) s[i] = dim[i + 1] > 1 ? (cuuint64_t)stride[i] * 2 : 128;
    return g_encode.load(std::memory_order_relaxed)(map, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5,
                    const_cast<void *>(base), d, s, b, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool F16>
cudaError_t launch(const AttnKernelParams &k, int ctas, cudaStream_t stream) {
    cudaError_t e = launch_kernel(attend<D, F16>, dim3((unsigned)ctas), kAttnThreads, Shape<D>::kSmem, stream, 0, true, k);
    if (e != cudaSuccess) return e;
    // as many blocks as an SM holds at most, and no more than there are rows for
    constexpr int R = kCombineThreads / (D / 4);
    const int64_t jobs = ((int64_t)k.p.num_tokens * k.p.hq + R - 1) / R;
    const Parts &parts = k;
    const JoinParams join = {k.p.out, k.p.lse, k.p.o_ts, k.p.o_hs, k.p.hq, k.p.group};
    return launch_kernel(combine<D, F16>, dim3((unsigned)std::min<int64_t>(8 * ctas, jobs)), kCombineThreads, 0, stream, 0,
                         true, parts, join, ctas);
}

constexpr size_t kStarterBytes = kAttnCtas * (sizeof(int4) + sizeof(int4));  // starters, then tails
constexpr size_t kMlBytes = 2 * (size_t)kAttnCtas * 2 * kTile * sizeof(float);

}  // namespace

size_t attn_workspace_bytes(int head_dim) {
    return kStarterBytes + kMlBytes + 2 * (size_t)kAttnCtas * kTile * (size_t)head_dim * sizeof(float);
}

int attn_max_requests() { return kMaxRequests; }

cudaError_t launch_tree_attention(const AttnParams &p, void *workspace, cudaStream_t stream) {
    int ctas;
    const cudaError_t e = prepare(&ctas);
    if (e != cudaSuccess) return e;
    AttnKernelParams k;
    k.p = p;
    unsigned char *ws = static_cast<unsigned char *>(workspace);
    k.starters = reinterpret_cast<int4 *>(ws);
    k.tails = reinterpret_cast<int *>(ws + kAttnCtas * sizeof(int4));
    k.ml = reinterpret_cast<float *>(ws + kStarterBytes);
    k.part = reinterpret_cast<float *>(ws + kStarterBytes + kMlBytes);

    // Pages.  A box of several 8-row groups must land as the tile holds them
    // (both 64-column halves of a group side by side), which takes the page
    // axis and the head axis (or the group axis) as one dimension: possible
    // when pages follow one another without gaps.  Other strides take 8 rows a
    // box.
    const int64_t D = p.d, H = p.hkv, ps = p.page_size, P = p.num_pages, halves = D / 64;
    const int br = (int)(ps < kTile ? ps : kTile);
    const bool small = P * H <= INT32_MAX / 2 && P * (ps / 8) <= INT32_MAX / 2;
    bool ok = true;
    const uint16_t *pools[2] = {p.k_pages, p.v_pages};
    CUtensorMap *whole[2] = {&k.maps.k, &k.maps.v}, *eight[2] = {&k.maps.k8, &k.maps.v8}, *fresh[2] = {&k.maps.kn, &k.maps.vn};
    const uint16_t *rows[2] = {p.k_new, p.v_new};
    if (small && p.page_stride == H * p.head_stride) k.form = kPagesHeadsOut;
    else if (small && p.page_stride == ps * p.token_stride) k.form = kPagesHeadsIn;
    else k.form = kPagesGeneral;
    k.box_groups = k.form == kPagesGeneral ? 1 : br / 8;
    for (int i = 0; i < 2; ++i) {
        ok = ok && encode(eight[i], pools[i], p.f16, {64, ps, halves, H, P},
                          {p.token_stride, 64, p.head_stride, p.page_stride}, {64, 8, (int)halves, 1, 1});
        if (k.form == kPagesHeadsOut)
            ok = ok && encode(whole[i], pools[i], p.f16, {64, 8, halves, ps / 8, P * H},
                              {p.token_stride, 64, 8 * p.token_stride, p.head_stride}, {64, 8, (int)halves, br / 8, 1});
        else if (k.form == kPagesHeadsIn)
            ok = ok && encode(whole[i], pools[i], p.f16, {64, 8, halves, H, P * (ps / 8)},
                              {p.token_stride, 64, p.head_stride, 8 * p.token_stride}, {64, 8, (int)halves, 1, br / 8});
        else
            *whole[i] = *eight[i];
        ok = ok && encode(fresh[i], rows[i], p.f16, {64, p.num_tokens, halves, H, 1}, {p.n_ts, 64, p.n_hs, 64},
                          {64, 8, (int)halves, 1, 1});
    }
    if (!ok) return cudaErrorInvalidValue;
    if (D == 64) return p.f16 ? launch<64, true>(k, ctas, stream) : launch<64, false>(k, ctas, stream);
    return p.f16 ? launch<128, true>(k, ctas, stream) : launch<128, false>(k, ctas, stream);
}

}  // namespace csgmv
