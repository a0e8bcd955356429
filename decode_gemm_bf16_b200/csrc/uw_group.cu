// uw_group.cu -- products of ragged groups of rows on the 5th-generation
// tensor cores: Y[s, n] = sum_k X[row(s), k] W[e(s), n, k], where expert e owns
// the slots offsets[e] .. offsets[e+1]-1, with W in BF16 or in the microscaled
// 4-bit form (MXFP4); optionally silu(X.W^T) * (X.U^T) from two weights.  One
// group is the plain MXFP4 product (BF16 or MXFP4 activations).
//
// Mathematics and bound.  A group of m rows costs 2 m N K operations and N K
// weight reads: below about 250 rows (BF16; 70 for 4-bit weights) it is bound
// by reading the weights of the experts that have rows, above by the tensor
// cores.  One kernel serves the range:
//   * swap-AB: 128 weight rows are the MMA's M, up to 256 slots of one expert
//     its N.  N is taken per tile (the tile's rows rounded up to 16), so a
//     ragged tail costs what it holds.  With `up`, 64 rows of each matrix
//     share the 128 (one pass over X, same MMA shape);
//   * tiles are listed on the device from the offsets: expert by expert, in
//     bands of 16 slot tiles with the slot tile fastest, so that CTAs working
//     at the same time share weight tiles and slot tiles in L2;
//   * one persistent CTA per SM, in pairs (cta_group::2: one MMA over 256 weight
//     rows) where tiles are large.  Full rounds of whole tiles are dealt out one
//     a worker; what is left over is cut along k where that pays (uw_plan.h).  The worker with a
//     cut tile's first k steps adds the others' fp32 partial sums in k order
//     (from the workspace; deterministic);
//   * warp roles: 0-7 epilogue, 8 and 11 TMA producers of weights and of X, 9 MMA
//     issue (10 and 12: see kMix; 12-19: see kGroupMx);
//   * 4-bit weights with BF16 rows (kGroupMx8): the tensor cores take the codes
//     and scales as they are, against 8-bit rows.  A BF16 value has 8
//     significant bits, an e4m3 value 4: x = 2^s (hi + lo/16) with both in
//     e4m3 and 2^s the scale of its block of 32 is exact for every x of at
//     least 2^-13 times the block's largest, and off by at most 2^-21 (1 + 2^-8)
//     of that largest below.  hi and lo are two rows of the MMA's N, added in fp32 at
//     the end: the operations of a BF16 product at twice the rate, and no
//     rebuilt weights.  A first kernel (k_group_split) writes the rows of
//     every tile in the order of its stages' shared memory, gathered, split
//     and swizzled, so a stage's rows and scales are one bulk copy; for pairs
//     with `up` it also joins the scales of the two weights;
//   * K an odd multiple of 64 (kGroupMx): the TMA's unpacking load wants rows
//     of 128 codes, so warps 12-19 rebuild codes to BF16 in tensor memory, the
//     MMA's A operand;
//   * MXFP4 with MXFP4 rows (kGroupMxMx): block-scaled 4-bit MMA; the scale
//     bytes go from shared to tensor memory (tcgen05.cp) in the order the
//     format stores them;
//   * gathered BF16 rows: tiles of up to 32 slots take them by TMA (four row
//     indices a request), larger ones from a gathered copy (k_group_gather):
//     a request of four rows of 128 bytes takes about 34 cycles, so 256 rows a
//     stage would take four times as long as the stage's MMAs;
//   * after one of these two kernels the weights of the first stages are
//     requested before the wait on it: it lets this kernel start only after
//     its own wait, so everything it does not write is complete;
//   * every wait is bounded; on expiry the CTA raises UW_ERR_TIMEOUT, drains
//     its own copies and MMAs, frees tensor memory and returns.
//
// Measured (one B200, GPU time alone, copy bandwidth 6.5 TB/s, library BF16
// product 1.63 PFLOP/s for a burst, 1.39 held):
//   BF16, gate and up of 8 experts of 14336 x 4096, 16 slots: 278 us, 6.8 TB/s
//     of weights;
//   BF16, 8 experts of 800-1493 rows, 4096 x 14336: 740 us, 1.30 PFLOP/s (1.11
//     held: the power limit), tensor pipe 96 % active; one group of 8192 rows
//     630 us, 1.53 (1.30 held, where the library's product has 1.31);
//   4-bit weights, 128 experts of 768 x 2048 twice, 264 slots: 49 us, 3.9 TB/s
//     of weights; 8 experts of 14336 x 4096 twice, 16 slots: 97 us, 5.1 TB/s;
//   4-bit weights, 64 experts of 1408 x 2048 twice, 12288 slots: 151-154 us, 0.93
//     PFLOP/s (25 us of it the split rows and joined scales); 2048 rows of 14336 x
//     4096: 171 us, 1.41 PFLOP/s; 4096 tokens of 2 of 8 experts of that shape
//     twice: 1346 us, 1.43 PFLOP/s (BF16 weights 1328, 1.45);
//   K an odd multiple of 64, 14336 x 4160: one row 33 us, 0.9 TB/s of weights;
//     2048 rows 207 us, 1.18 PFLOP/s;
//   both in 4 bits, 2048 rows of 14336 x 4096: 52 us, 4.7 PFLOP/s, one row 12-13
//     us; 8192^3: 192 us, 5.7 PFLOP/s.
#include <cuda_fp16.h>
#include <cstdlib>

#include "uw_device.cuh"
#include "uw_internal.h"
#include "uw_plan.h"

namespace uw {

int group_status_take() { return unit_status_take(); }

namespace {

constexpr int kTileN = 128;            // weight rows of a tile
constexpr int kProd = 8, kMma = 9, kRebuild0 = 12, kRebuildWarps = 8;
constexpr int kEpiWarps = 8;           // two per quarter of tensor memory's lanes
constexpr int kMix = 10, kMix2 = 12;    // kGroupMx8, single CTAs: warps that join the scales of two weights, every other slot each
constexpr int kRows = 11;              // TMA producer of X
constexpr int kThreadsPlain = 12 * 32, kThreadsMix = 13 * 32;
constexpr int kThreadsRebuild = (kRebuild0 + kRebuildWarps) * 32;
constexpr int kMaxS = 12;              // stages
constexpr int kMaxT = 8;               // rebuilt-A slots in tensor memory
constexpr int kBand = 16;              // slot tiles of a band
constexpr int kEpiBarId = 1;
constexpr uint32_t kWarpStage = 2048;  // transpose buffer of an epilogue warp
constexpr uint32_t kExchange = kEpiWarps * 2048;   // `up`: 16 slots x 32 rows of fp32 sums a warp
constexpr uint32_t kTmemCols = 512;
constexpr uint64_t kRestNs = 1000000;  // after an expired wait: see the kernel's end

// Tensor maps of a call (unused ones are left empty).
struct Maps {
    CUtensorMap x;        // rows of X (or, split rows, 16 prepared rows a box)
    CUtensorMap w, u;     // weights
    CUtensorMap sw;       // W's scale tiles, or the joined ones of W and `up`, 512 bytes a row (pairs)
    CUtensorMap sx;       // X's (pairs; split rows: the scales in front of the prepared rows)
};

struct GroupParams {
    int64_t x_rows, slots, N;
    const int32_t* rows;
    const int32_t* offsets;
    int E, kt, MG, box, n_tiles, up, out_f32, y_vec;
    int S, T, nacc;
    uint32_t acc_w;                         // columns of an accumulator
    uint32_t stage_bytes, off_s, off_b;     // codes (or BF16 weights) at 0, scale bytes, X
    uint32_t sf_a_bytes, sf_b_bytes;        // scale bytes of a stage: weights (one matrix), X
    uint32_t sf_slot;                       // scale columns of a stage
    uint32_t a_col0, sf_col0;
    int step;                               // tiles of a group hold a multiple of this many slots
    int parts;                              // cut tiles in equal parts (uw_plan.h)
    int early;                              // a preparing kernel of this call ran just before
    const uint8_t* prep;                    // kGroupMx8: [slot tiles][kt][scales, rows]
    int64_t prep_chunk;                     // bytes of one stage of one tile there
    int part_f4;                            // float4 columns of a partial row
    uint32_t ctrl_off, stg_off, tab_off, work_off;
    const uint8_t* sw;                      // scale tiles of W, up
    const uint8_t* su;
    int64_t w_row_tiles;                    // scale row tiles of one matrix
    int k_tiles;                            // scale tiles along k
    void* Y;
    float* partial;                         // [CTAs][MG/4][128] float4
    unsigned long long* flags;              // [CTAs][8]: call tag once a warp's partial sums are out
    unsigned long long epoch;
    unsigned long long tag;                 // what is written there: the epoch (but for a test of the limit)
    uint64_t timeout;
};

struct Ring {
    int i = 0;
    uint32_t ph = 0;
    __device__ __forceinline__ void advance(int n) {
        if (++i == n) {
            i = 0;
            ph ^= 1u;
        }
    }
};

// The tile list as every role sees it (shared memory).
struct Tiles {
    const int32_t* cum;      // [E + 1] tiles before each expert
    const int32_t* begin;    // [E] first slot
    const int32_t* count;    // [E] slots
};

// Slots of a tile of a group of c: the group is cut into as few tiles of at
// most MG slots as it takes, all of one size but the last (a multiple of
// `step`, so never more than MG).  Even tiles keep the workers of a round in
// step; a short last tile would let its worker run ahead (8 uneven experts
// of 800-1493 rows, 4096 x 14336 in BF16: 804 us with tiles of 256 and a rest,
// 736 us).
__device__ __forceinline__ int tile_slots(int c, int MG, int step) {
    const int mt = (c + MG - 1) / MG, even = (c + mt - 1) / mt;
    return (even + step - 1) / step * step;
}

struct Tile {
    int e, n, rows;          // expert, weight tile, slots of the tile
    int64_t s0;              // first slot
    int64_t m;               // the slot tile's number among all
};

// A worker's segments with their tiles.  The first kListed are worked out by
// the block's threads at once when it starts (in every role, one after the
// other, they cost 1700 cycles a tile).
constexpr int kListed = 40;
struct Work {
    Seg seg;
    Tile tile;
};

__device__ __forceinline__ Tile locate(const GroupParams& p, const Tiles& tl, uint32_t utile) {
    const int tile = (int)utile;   // below 2^31
    int lo = 0, hi = p.E;   // last expert with cum[e] <= tile (experts without tiles are passed over)
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (tl.cum[mid] <= tile) lo = mid; else hi = mid;
    }
    const int c = tl.count[lo];
    const int mt = (c + p.MG - 1) / p.MG;
    int l = tile - tl.cum[lo];
    const int band = l / (kBand * p.n_tiles);
    l -= band * kBand * p.n_tiles;
    const int nb = mt - band * kBand < kBand ? mt - band * kBand : kBand;
    Tile t;
    t.e = lo;
    t.n = l / nb;
    const int m = band * kBand + l % nb;
    const int each = tile_slots(c, p.MG, p.step);
    t.s0 = (int64_t)tl.begin[lo] + (int64_t)m * each;
    t.m = tl.cum[lo] / p.n_tiles + m;
    t.rows = c - m * each < each ? c - m * each : each;
    return t;
}

struct Walk {
    const Work* list;
    int worker, i = 0;
    __device__ __forceinline__ Walk(const Work* l, int b) : list(l), worker(b) {}
    __device__ __forceinline__ bool next(const GroupParams& p, const Tiles& tl, const Plan& pl, Seg& s, Tile& t) {
        if (i < kListed) {
            s = list[i].seg;
            t = list[i].tile;
            i++;
            return t.rows > 0;
        }
        if (!segment(pl, (uint32_t)worker, (uint32_t)i, s)) return false;
        i++;
        t = locate(p, tl, s.tile);
        return true;
    }
};

__device__ __forceinline__ uint32_t bf2(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// g / (1 + e^-g).  The fast division gives 0 for denominators above 2^126; a
// quarter of either side keeps the largest finite one at 2^126.  (An exact
// division: 128 experts of 768 x 2048 twice in 4 bits, 264 slots, 50.7 us, so 49.4.)
__device__ __forceinline__ float silu(float g) { return __fdividef(0.25f * g, fmaf(0.25f, __expf(-g), 0.25f)); }

// Y[s0 + i, nw + lane] = v[i] for 16 slots (`valid` of them in the tile), by a
// whole warp.  A lane holds one output of 16 slots; written so, a warp's
// store would put 2 bytes a lane into 16 rows.  Instead slots go in pairs of
// BF16 through 1 KB of shared memory and leave as 16-byte stores, four lanes a
// slot.  Rows of N values that are not 16-byte aligned (N % 8) are stored value
// by value, and so is fp32 (128 contiguous bytes a slot already).
__device__ __forceinline__ void put_plain(const GroupParams& p, const uint32_t (&v)[16], int64_t s0, int valid, int64_t nw, int lane) {
    if (nw + lane >= p.N) return;
    const int64_t at = s0 * p.N + nw + lane;
#pragma unroll
    for (int i = 0; i < 16; i++)
        if (i < valid) {
            if (p.out_f32) reinterpret_cast<float*>(p.Y)[at + i * p.N] = __uint_as_float(v[i]);
            else reinterpret_cast<__nv_bfloat16*>(p.Y)[at + i * p.N] = __float2bfloat16_rn(__uint_as_float(v[i]));
        }
}
__device__ __forceinline__ void stage16(const uint32_t (&v)[16], int lane, uint32_t stg) {
#pragma unroll
    for (int i = 0; i < 8; i++) sts32(stg + (uint32_t)(i * 128 + lane * 4), bf2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])));
}
// (lane: slots 2 (lane / 4) and the next, outputs 8 (lane % 4) ..)
__device__ __forceinline__ void put16(const GroupParams& p, int64_t s0, int valid, int64_t nw, int lane, uint32_t stg) {
    const int s = (lane >> 2) * 2, o = (lane & 3) * 8;
    const uint4 a = lds128(stg + (uint32_t)((lane >> 2) * 128 + (lane & 3) * 32));
    const uint4 b = lds128(stg + (uint32_t)((lane >> 2) * 128 + (lane & 3) * 32 + 16));
    if (nw + o >= p.N) return;
    uint16_t* y = reinterpret_cast<uint16_t*>(p.Y) + (s0 + s) * p.N + nw + o;
    if (s < valid)
        *reinterpret_cast<uint4*>(y) = make_uint4(prmt(a.x, a.y, 0x5410u), prmt(a.z, a.w, 0x5410u), prmt(b.x, b.y, 0x5410u), prmt(b.z, b.w, 0x5410u));
    if (s + 1 < valid)
        *reinterpret_cast<uint4*>(y + p.N) =
            make_uint4(prmt(a.x, a.y, 0x7632u), prmt(a.z, a.w, 0x7632u), prmt(b.x, b.y, 0x7632u), prmt(b.z, b.w, 0x7632u));
}
__device__ __forceinline__ void store16(const GroupParams& p, const uint32_t (&v)[16], int64_t s0, int valid, int64_t nw, int lane,
                                        uint32_t stg) {
    if (p.out_f32 || !p.y_vec) {
        put_plain(p, v, s0, valid, nw, lane);
        return;
    }
    __syncwarp();   // the buffer's last readers are through
    stage16(v, lane, stg);
    __syncwarp();
    put16(p, s0, valid, nw, lane, stg);
}
// 32 slots (16 unless `two`) in one go.
__device__ __forceinline__ void store32(const GroupParams& p, const uint32_t (&v)[2][16], bool two, int64_t s0, int valid, int64_t nw,
                                        int lane, uint32_t stg) {
    if (p.out_f32 || !p.y_vec) {
        put_plain(p, v[0], s0, valid, nw, lane);
        if (two) put_plain(p, v[1], s0 + 16, valid - 16, nw, lane);
        return;
    }
    __syncwarp();
    stage16(v[0], lane, stg);
    if (two) stage16(v[1], lane, stg + 1024u);
    __syncwarp();
    put16(p, s0, valid, nw, lane, stg);
    if (two) put16(p, s0 + 16, valid - 16, nw, lane, stg + 1024u);
}

__device__ __forceinline__ bool any_of_epilogue(bool pred) {
    uint32_t res;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "bar.red.or.pred q, %2, %3, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(res)
        : "r"((uint32_t)pred), "n"(kEpiBarId), "n"(kEpiWarps * 32)
        : "memory");
    return res != 0;
}

// Four rows of X by index (box one row high) into 4 consecutive 128-byte rows.
__device__ __forceinline__ void tma_gather4(uint32_t dst, const CUtensorMap* map, int x, int4 r, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cta.global.tile::gather4.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
        "l"(map), "r"(x), "r"(r.x), "r"(r.y), "r"(r.z), "r"(r.w), "r"(bar)
        : "memory");
}

// 512 bytes of scales (32 rows x 16 bytes) at shared address 16 * (smem16 %
// 2^14) -> 4 columns of tensor memory, in every quarter of the lanes.
template <int CG>
__device__ __forceinline__ void tc_copy_scales(uint32_t tmem, uint32_t smem16) {
    // rows of 16 bytes in 8-row groups of 128 bytes, no swizzle
    const uint64_t d = ((uint64_t)((128u >> 4) | (1u << 14)) << 32) | (smem16 & 0x3FFFu);
    if (CG == 1) asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(d) : "memory");
    else asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(d) : "memory");
}

// D (+)= A * B^T with e2m1 operands and one e8m0 scale per 32 k (K = 64), by a pair.
__device__ __forceinline__ void tc_mma_mx(uint32_t d_tmem, uint64_t ad, uint64_t bd, uint32_t idesc, uint32_t sfa,
                                          uint32_t sfb, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d_tmem),
        "l"(ad), "l"(bd), "r"(idesc), "r"(sfa), "r"(sfb), "r"(acc)
        : "memory");
}

template <int CG>
__device__ __forceinline__ void tc_mma_bf16(uint32_t d_tmem, uint64_t ad, uint64_t bd, uint32_t idesc, uint32_t acc) {
    if (CG == 1)
        tc_mma(d_tmem, ad, bd, idesc, acc);
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
            "l"(ad), "l"(bd), "r"(idesc), "r"(acc)
            : "memory");
}

// Instruction descriptor of kind::mxf4: both operands e2m1, scales e8m0, both
// K-major, M = 128 a CTA; `id` (0 or 2) picks the scale bytes' half word.
__device__ __forceinline__ uint32_t idesc_mx(int CG, int N, uint32_t id) {
    return (id << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | (1u << 23) | ((uint32_t)CG << 27) | (id << 29);
}

// 32 codes with scale byte s -> 16 BF16 pairs.  The eight magnitudes times
// 2^s come first (four packed multiplications, exact: a power of two), split
// into a table of low and one of high bytes; each code then picks its bytes by
// permute, and its sign enters the high byte.
__device__ __forceinline__ void rebuild32(const uint4 c, uint32_t s, uint32_t (&out)[16]) {
    const uint32_t f1 = s == 255u ? 0x7FC0u : s ? s << 7 : 0x0040u;
    const uint32_t f = f1 | (f1 << 16);
    const uint32_t mags[4] = {0x3F000000u, 0x3FC03F80u, 0x40404000u, 0x40C04080u};   // 0 .5 | 1 1.5 | 2 3 | 4 6
    uint32_t m[4];
#pragma unroll
    for (int i = 0; i < 4; i++) asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(m[i]) : "r"(mags[i]), "r"(f));
    const uint32_t L0 = prmt(m[0], m[1], 0x6420u), L1 = prmt(m[2], m[3], 0x6420u);
    const uint32_t H0 = prmt(m[0], m[1], 0x7531u), H1 = prmt(m[2], m[3], 0x7531u);
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const uint32_t mag = w[i] & 0x77777777u;
        const uint32_t t = w[i] & 0x88888888u;
        const uint32_t sg = t | (t >> 1);   // nibble 0xC (the sign of byte 4, 0x80, replicated) or 0
#pragma unroll
        for (int h = 0; h < 2; h++) {
            const uint32_t sel = h ? mag >> 16 : mag, ss = h ? sg >> 16 : sg;
            const uint32_t lo = prmt(L0, L1, sel);
            const uint32_t hi = prmt(H0, H1, sel) | (prmt(0u, 0x80u, ss) & 0x80808080u);
            out[4 * i + 2 * h] = prmt(lo, hi, 0x5140u);
            out[4 * i + 2 * h + 1] = prmt(lo, hi, 0x7362u);
        }
    }
}

// 16-byte chunk c of row r in rows of 32 bytes stored with the 32-byte swizzle.
__device__ __forceinline__ uint32_t sw32(int r, int c) { return r * 32 + ((c ^ ((r >> 2) & 1)) << 4); }

// D (+)= A * B^T, A e2m1 (a byte each), B e4m3, one e8m0 scale per 32 k (K = 32).
template <int CG>
__device__ __forceinline__ void tc_mma_mx8(uint32_t d_tmem, uint64_t ad, uint64_t bd, uint32_t idesc, uint32_t sfa,
                                           uint32_t sfb, uint32_t acc) {
    if (CG == 1)
        asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d_tmem),
        "l"(ad), "l"(bd), "r"(idesc), "r"(sfa), "r"(sfb), "r"(acc)
        : "memory");
    else
        asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d_tmem),
        "l"(ad), "l"(bd), "r"(idesc), "r"(sfa), "r"(sfb), "r"(acc)
        : "memory");
}

// Instruction descriptor of kind::mxf8f6f4: A e2m1, B e4m3, scales e8m0, both
// K-major, M = 128 a CTA; `id` (0..3) picks the scale byte.
__device__ __forceinline__ uint32_t idesc_mx8(int CG, int N, uint32_t id) {
    return (id << 4) | (5u << 7) | ((uint32_t)(N >> 3) << 17) | (1u << 23) | ((uint32_t)CG << 27) | (id << 29);
}

// Columns of the MMA's N for a tile of `rows` slots: the rows rounded up to
// 16; two of them (hi, lo) per row rounded up to 8 for split rows.  A pair
// takes multiples of 32, 16 a CTA.
template <int SRC, int CG>
__device__ __forceinline__ int mma_n(int rows) {
    constexpr int step = (SRC == kGroupMx8 ? 8 : 16) * CG;
    return (rows + step - 1) / step * step * (SRC == kGroupMx8 ? 2 : 1);
}

// The tile list from the offsets: tables cum[E + 1], begin[E], count[E] in
// shared memory.  Every thread of the block calls it (it synchronises twice);
// all offsets are loaded at once, then 32 runs of experts are summed by warp 0.
__device__ __forceinline__ void list_tiles(const int32_t* offsets, int E, int64_t slots, int MG, int n_tiles, int32_t* cum,
                                           int32_t* begin, int32_t* count) {
    const int tid = threadIdx.x, lane = tid & 31;
    bool bad = false;
    for (int e = tid; e < E; e += blockDim.x) {
        int64_t o0 = 0, o1 = slots;
        if (offsets) {
            o0 = offsets[e];
            o1 = offsets[e + 1];
        }
        const bool wrong = o0 < 0 || o1 < o0 || o1 > slots;
        bad |= wrong;
        begin[e] = wrong ? 0 : (int)o0;
        count[e] = wrong ? 0 : (int)(o1 - o0);
    }
    const int any = __syncthreads_or(bad);
    if (any && bad) raise_status(UW_ERR_DEVICE);
    if (tid < 32) {
        const int each = (E + 31) / 32, lo = lane * each < E ? lane * each : E, hi = lo + each < E ? lo + each : E;
        int sum = 0;
        for (int e = lo; e < hi; e++) sum += any ? 0 : (count[e] + MG - 1) / MG * n_tiles;   // falling or past the slots: no tiles at all
        int run = sum;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int v = __shfl_up_sync(0xFFFFFFFFu, run, d);
            if (lane >= d) run += v;
        }
        int at = run - sum;
        for (int e = lo; e < hi; e++) {
            cum[e] = at;
            at += any ? 0 : (count[e] + MG - 1) / MG * n_tiles;
        }
        if (lane == 31) cum[E] = run;
    }
    __syncthreads();
}

// k of a stage.
constexpr int stage_k(int src) { return src == kGroupMx8 ? 128 : src == kGroupMxMx ? 256 : 64; }

// ---- pairs of CTAs (cta_group::2): forms of the shared helpers
template <int CG>
__device__ __forceinline__ void pair_alloc(uint32_t dst, uint32_t cols) {
    if (CG == 1) {
        tmem_alloc(dst, cols);
        tmem_relinquish();
    } else {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst), "r"(cols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
}
template <int CG>
__device__ __forceinline__ void pair_dealloc(uint32_t taddr, uint32_t cols) {
    if (CG == 1) tmem_dealloc(taddr, cols);
    else asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(cols) : "memory");
}
// Arrive once on `bar` (of both CTAs of a pair) when the MMAs issued so far are done.
template <int CG>
__device__ __forceinline__ void pair_commit(uint32_t bar) {
    if (CG == 1)
        tc_commit(bar);
    else
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
                     "h"((uint16_t)3)
                     : "memory");
}
// Address of this CTA's `bar` in the pair's first CTA, and an arrival there.
__device__ __forceinline__ uint32_t in_first(uint32_t bar) {
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(a) : "r"(bar));
    return a;
}
// arrive_at orders no writes: it is for the accumulator's release alone, where
// there are none to order (see `release`).
__device__ __forceinline__ void arrive_at(uint32_t cluster_bar) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}
__device__ __forceinline__ bool test_cluster(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
// A box into this CTA's shared memory, counted on the barrier of the pair's
// first CTA (`bar`: its cluster address).
__device__ __forceinline__ void tma_load_pair(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
template <int CG>
__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
    if (CG == 1) tma_load_2d(dst, map, x, y, bar);
    else tma_load_pair(dst, map, x, y, bar);
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Wait of a role's single thread: one test where the phase is complete, the
// bounded wait out of line.
__device__ __noinline__ bool wait_slow(uint32_t bar, uint32_t parity, uint64_t timeout, volatile int* abort) {
    return mbar_wait(bar, parity, timeout, abort);
}
__device__ __forceinline__ bool wait_one(uint32_t bar, uint32_t parity, uint64_t timeout, volatile int* abort) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0 || mbar_try_wait(bar, parity, 1000) || wait_slow(bar, parity, timeout, abort);
}
// The same for a barrier on which the pair's other CTA arrives too.
template <int CG>
__device__ __forceinline__ bool wait_pair(uint32_t bar, uint32_t parity, uint64_t timeout, volatile int* abort) {
    if (CG == 1) return wait_one(bar, parity, timeout, abort);
    if (test_cluster(bar, parity)) return true;
    const uint64_t deadline = globaltimer() + timeout;
    for (uint32_t i = 1;; i++) {
        if (test_cluster(bar, parity)) return true;
        if ((i & 63u) == 0) {
            if (*abort) return false;
            if (globaltimer() > deadline) {
                *abort = 1;
                return false;
            }
        }
    }
}

// What the producer thread loads for the stages of one tile, from k step kt on:
// everything that changes from stage to stage is advanced, not computed anew.
// In a pair every load counts on the first CTA's barrier, which expects the
// bytes of both.
template <int SRC, int CG>
struct Feed {
    static constexpr int KB = stage_k(SRC);
    static constexpr uint32_t kARow = SRC == kGroupMx ? 32 : 128;
    const CUtensorMap* second;   // map of the tile's rows 64..127
    int ax, w0, w1;              // column and rows of the weight boxes
    const uint8_t* s0;           // scales of the stage's weights (and of `up`)
    const uint8_t* s1;
    int sy;                      // ... their half tile (pairs)
    int half;                    // kGroupMx: a scale half tile (128 k) serves two stages
    const uint8_t* x0;           // split rows
    int xy0, xy1;                // ... their row (pairs), or the half tile of the scales of 128 rows of X (and of the next 128)
    int bx, y, boxes, gathers;
    uint32_t x_bytes, tx;

    __device__ __forceinline__ Feed(const GroupParams& p, const Maps& m, const Tile& t, int kt, int rank) {
        const int n0 = (t.n * CG + rank) * (p.up ? kTileN / 2 : kTileN), nN = mma_n<SRC, CG>(t.rows) / CG;
        w0 = t.e * (int)p.N + n0;   // E N is below 2^31
        w1 = p.up ? w0 : w0 + kTileN / 2;
        second = p.up ? &m.u : &m.w;
        // codes that the TMA unpacks count as elements of a box, packed ones as bytes
        ax = kt * (SRC == kGroupBf16 || SRC == kGroupMx8 ? KB : KB / 2);
        bx = kt * (SRC == kGroupMxMx ? KB / 2 : KB);
        y = (int)t.s0 + rank * nN;
        boxes = (nN + p.box - 1) / p.box;
        gathers = CG == 1 && p.rows ? (t.rows + 3) / 4 : 0;
        x_bytes = SRC == kGroupMx8 && CG == 1 ? (uint32_t)nN * 128u : gathers ? (uint32_t)gathers * 512u : (uint32_t)(boxes * p.box) * 128u;
        // the unpacking load counts the packed bytes of its rows
        tx = (uint32_t)kTileN * (SRC == kGroupMx8 ? 64u : kARow) + p.sf_b_bytes + x_bytes;
        tx += p.sf_a_bytes * (p.up && CG == 1 ? 2u : 1u);
        tx *= CG;
        s0 = s1 = x0 = nullptr;
        sy = half = xy0 = xy1 = 0;
        if (SRC != kGroupBf16) {
            // the stage's part of a scale tile (256 k): all of it, or the half that holds the stage
            // (the second CTA of a pair may stand past the last row tile)
            const int64_t row_tile = n0 / kMxTileRows < p.w_row_tiles ? n0 / kMxTileRows : p.w_row_tiles - 1;
            const int64_t at = 2 * ((int64_t)t.e * p.w_row_tiles + row_tile) * p.k_tiles +
                               (SRC == kGroupMxMx ? 2 * kt : SRC == kGroupMx8 ? kt : kt >> 1);
            half = kt & 1;
            s0 = p.sw + at * (kMxTileBytes / 2);
            if (p.up) s1 = p.su + at * (kMxTileBytes / 2);
            sy = joined(p) ? (int)((2 * (t.e * p.w_row_tiles + t.n) + rank) * p.kt + kt) : (int)at;
        }
        if (SRC == kGroupMx8) {
            const int64_t chunk = t.m * p.kt + kt;
            x0 = p.prep + chunk * p.prep_chunk;
            xy0 = (int)(chunk * (p.prep_chunk / 128));
            xy1 = xy0 + (int)(p.sf_b_bytes / 128u) + rank * nN;
        }
        if (SRC == kGroupMxMx) {
            // a row tile past the last reads the last one again (rows past the end: never stored)
            const int64_t rt = t.s0 / kMxTileRows, last = (p.x_rows - 1) / kMxTileRows;
            const int64_t a0 = rt * p.k_tiles + kt, a1 = (rt < last ? rt + 1 : last) * p.k_tiles + kt;
            xy0 = (int)(2 * a0);
            xy1 = (int)(2 * a1);
        }
    }
    // scales of two weights, joined before this kernel: loaded with X, behind the wait for what the preparing kernel writes
    __device__ static __forceinline__ bool joined(const GroupParams& p) { return SRC == kGroupMx8 && CG == 2 && p.up; }

    // `lb`: the stage's barrier here, `fb`: the one that counts (pairs: the first CTA's)
    __device__ __forceinline__ void weights(const GroupParams& p, const Maps& m, uint32_t st, uint32_t lb, uint32_t fb, bool expect) {
        if (expect) mbar_arrive_expect_tx(lb, tx);
        load_box<CG>(st, &m.w, ax, w0, fb);
        load_box<CG>(st + kTileN / 2 * kARow, second, ax, w1, fb);
        ax += SRC == kGroupBf16 || SRC == kGroupMx8 ? KB : KB / 2;
        if (SRC != kGroupBf16) {
            if (CG == 1) {
                bulk_load(st + p.off_s, s0, p.sf_a_bytes, fb);
                if (p.up) bulk_load(st + p.off_s + p.sf_a_bytes, s1, p.sf_a_bytes, fb);
            } else if (!joined(p)) {
                tma_load_pair(st + p.off_s, &m.sw, 0, sy, fb);
            }
            const uint32_t step = SRC == kGroupMx && !half ? 0 : p.sf_a_bytes;
            s0 += step;
            s1 += step;
            sy += SRC == kGroupMxMx ? 2 : 1;
            if (SRC == kGroupMx) half ^= 1;
        }
    }
    __device__ __forceinline__ void rows(const GroupParams& p, const Maps& m, uint32_t st, uint32_t fb, const int4 (&idx)[8]) {
        if (SRC == kGroupMx8) {
            if (CG == 1) {   // scales and rows, one run in both memories
                bulk_load(st + p.off_b - p.sf_b_bytes, x0, p.sf_b_bytes + x_bytes, fb);
                x0 += p.prep_chunk;
            } else {         // all columns' scales, this CTA's half of the rows
                if (p.up) tma_load_pair(st + p.off_s, &m.sw, 0, sy++, fb);
                tma_load_pair(st + p.off_b - p.sf_b_bytes, &m.sx, 0, xy0, fb);
                for (int b = 0; b < boxes; b++) tma_load_pair(st + p.off_b + (uint32_t)(b * p.box) * 128u, &m.x, 0, xy1 + b * p.box, fb);
                xy0 += (int)(p.prep_chunk / 128);
                xy1 += (int)(p.prep_chunk / 128);
            }
            return;
        }
        if (SRC == kGroupMxMx) {
            tma_load_pair(st + p.off_b - p.sf_b_bytes, &m.sx, 0, xy0, fb);
            if (p.sf_b_bytes > kMxTileBytes) tma_load_pair(st + p.off_b - kMxTileBytes, &m.sx, 0, xy1, fb);
            xy0 += 2;
            xy1 += 2;
        }
        if (gathers) {
#pragma unroll
            for (int g = 0; g < 8; g++)
                if (g < gathers) tma_gather4(st + p.off_b + (uint32_t)g * 512u, &m.x, bx, idx[g], fb);
        } else {
            for (int b = 0; b < boxes; b++) load_box<CG>(st + p.off_b + (uint32_t)(b * p.box) * 128u, &m.x, bx, y + b * p.box, fb);
        }
        bx += SRC == kGroupMxMx ? KB / 2 : KB;
    }
};

template <int SRC, int CG>
__device__ __forceinline__ void group_body(const Maps& m, const GroupParams& p) {
    static_assert(SRC != kGroupMxMx || CG == 2, "4-bit rows take tiles of 128 slots at least: always pairs (pick_pair)");
    constexpr int KB = stage_k(SRC);
    constexpr bool kRe = SRC == kGroupMx;
    constexpr bool kScaled = SRC == kGroupMx8 || SRC == kGroupMxMx;   // scales in tensor memory
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    uint8_t* smem = smem_raw + (base - smem_u32(smem_raw));
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + p.ctrl_off);
    const uint32_t full = smem_u32(bars), empty = full + 8 * kMaxS, recon = empty + 8 * kMaxS, tfree = recon + 8 * kMaxT;
    const uint32_t accf = tfree + 8 * kMaxT, acce = accf + 16, fin = acce + 16, mixed = fin + 8;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 3 * kMaxS + 2 * kMaxT + 5);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    int32_t* cum = reinterpret_cast<int32_t*>(smem + p.tab_off);
    int32_t* begin = cum + p.E + 1;
    int32_t* count = begin + p.E;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // A pair of CTAs works as one on 256 weight rows: each holds its 128 rows
    // and half of the tile's X; the first issues the MMAs of both.
    // Workers count down with the block index: whoever joins a tile's parts
    // waits for higher workers, that is for blocks that started before it, so
    // the wait ends even where not all blocks are resident at once, and blocks
    // that start late, behind the kernel before, are the ones that wait anyway
    // (300 rows, 4096 x 14336 in BF16: 45 us; counting up, 58).
    const int rank = CG == 2 ? (int)(blockIdx.x & 1) : 0, worker = (int)((gridDim.x - 1 - blockIdx.x) / CG);

    if (warp == 0) {   // a lane a barrier of each kind
        if (lane < p.S) {
            mbar_init(full + 8 * lane, 1);
            mbar_init(empty + 8 * lane, 1);
            mbar_init(mixed + 8 * lane, 1);
        }
        if (kRe && lane < p.T) {
            mbar_init(recon + 8 * lane, kRebuildWarps);
            mbar_init(tfree + 8 * lane, 1);
        }
        if (lane < 2) {
            mbar_init(accf + 8 * lane, 1);
            mbar_init(acce + 8 * lane, kEpiWarps * CG);
        }
        if (lane == 0) {
            mbar_init(fin, 1);
            *abort_flag = 0;
        }
        fence_barrier_init();
    }
    if (warp == kMma) pair_alloc<CG>(smem_u32(tmem_slot), kTmemCols);
    if (warp == kProd && lane == 0) {
        tma_prefetch_desc(&m.w);
        if (p.up) tma_prefetch_desc(&m.u);
        if (SRC != kGroupMx8 || CG == 2) tma_prefetch_desc(&m.x);
    }
    // With a preparing kernel before this one the offsets and weights are
    // complete already (see k_group_split); what it writes is waited for below.
    if (!p.early) asm volatile("griddepcontrol.wait;" ::: "memory");
    // By the warp that allocates, once it has: a dependent CTA on the same SM that took the tensor memory first would keep
    // it while it waits for this kernel.  (By all warps after the table below: 64 rows of 14336 x 4096 17.7 us, so 16.7.)
    if (warp == kMma) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    tc_fence_before();
    list_tiles(p.offsets, p.E, p.slots, p.MG, p.n_tiles, cum, begin, count);
    if (CG == 2) cluster_sync();   // both CTAs' barriers are there
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    const Tiles tl{cum, begin, count};
    const Plan pl = make_plan((uint32_t)cum[p.E], gridDim.x / CG, (uint32_t)p.kt, p.acc_w, p.parts != 0);
    Work* work = reinterpret_cast<Work*>(smem + p.work_off);
    for (int i = threadIdx.x; i < kListed; i += blockDim.x) {
        Work w;
        if (segment(pl, (uint32_t)worker, (uint32_t)i, w.seg)) w.tile = locate(p, tl, w.seg.tile);
        else w.tile.rows = 0;
        work[i] = w;
    }
    __syncthreads();
    // (the weights' producer goes ahead: everything it reads is complete)
    if (p.early && warp != kProd) asm volatile("griddepcontrol.wait;" ::: "memory");
    const int rows_a = p.up ? kTileN / 2 : kTileN;   // outputs of a tile

    if (warp == kProd) {
        // ------------------------------------------------------------ TMA producer: weights and their scales
        // One thread walks the stages.  X has a thread of its own (below): one
        // thread for both took 500 cycles a stage of 4-bit weights, more than
        // its MMAs, and 1700 where the tile changes.
        if (elect_one()) {
            Walk wk(work, worker);
            Seg sg;
            int slot = 0;
            int64_t q = 0;
            uint32_t ph = 1, st = base, fb = full;
            const uint32_t sig = CG == 2 ? in_first(full) - full : 0;   // from a barrier here to the first CTA's
            bool ok = true;
            Tile t;
            while (ok && wk.next(p, tl, pl, sg, t)) {
                Feed<SRC, CG> f(p, m, t, sg.kt0, rank);
                for (int kt = sg.kt0; kt < sg.kt1; kt++, q++) {
                    if (!wait_one(fb + 8 * kMaxS, ph, p.timeout, abort_flag)) { ok = false; break; }   // empty
                    f.weights(p, m, st, fb, fb + sig, rank == 0);
                    st += p.stage_bytes;
                    fb += 8;
                    if (++slot == p.S) {
                        slot = 0;
                        ph ^= 1u;
                        st = base;
                        fb = full;
                    }
                }
            }
            // The MMAs' last commits arrive on barriers of both CTAs of a pair, and the second CTA would not wait for
            // them otherwise: a CTA that left first would have them reach shared memory that it no longer owns.  So the
            // ring is walked once more (a slot never used passes at once), then the final commit is waited for.
            for (int i = 0; ok && i < p.S; i++) {
                ok = wait_one(fb + 8 * kMaxS, ph, p.timeout, abort_flag);
                fb += 8;
                if (++slot == p.S) {
                    slot = 0;
                    ph ^= 1u;
                    fb = full;
                }
            }
            if (rank) mbar_wait(fin, 0, 4 * p.timeout, nullptr);   // (the first CTA commits it on every path)
            // On expiry the loads of the last stages land before the CTA (or the pair) exits.  (All of them within one
            // limit: a stage of which another thread issued no part never completes.)
            if (!ok && rank == 0) {
                const uint64_t end = globaltimer() + p.timeout;
                for (int64_t qq = q - p.S < 0 ? 0 : q - p.S; qq < q; qq++) {
                    const uint64_t t0 = globaltimer();
                    mbar_wait(full + 8 * (uint32_t)(qq % p.S), (uint32_t)((qq / p.S) & 1), t0 < end ? end - t0 : 0, nullptr);
                }
            }
        }
        __syncwarp();
    } else if (warp == kRows) {
        // ------------------------------------------------------------ TMA producer: X
        if (elect_one()) {
            Walk wk(work, worker);
            Seg sg;
            int slot = 0;
            uint32_t ph = 1, st = base, fb = full;
            const uint32_t sig = CG == 2 ? in_first(full) - full : 0;
            bool ok = true;
            Tile t;
            while (ok && wk.next(p, tl, pl, sg, t)) {
                Feed<SRC, CG> f(p, m, t, sg.kt0, rank);
                int4 idx[8];
                if (CG == 1 && p.rows) {
                    // four rows a request; past the tile's end its last row again (never stored)
                    int* ip = &idx[0].x;
                    bool wrong = false;
#pragma unroll
                    for (int i = 0; i < 32; i++) {
                        const int32_t v = p.rows[t.s0 + (i < t.rows ? i : t.rows - 1)];
                        const bool in = v >= 0 && v < p.x_rows;
                        wrong |= !in;
                        ip[i] = in ? v : 0;
                    }
                    if (wrong) raise_status(UW_ERR_DEVICE);
                }
                for (int kt = sg.kt0; kt < sg.kt1; kt++) {
                    if (!wait_one(fb + 8 * kMaxS, ph, p.timeout, abort_flag)) { ok = false; break; }   // empty
                    f.rows(p, m, st, fb + sig, idx);
                    st += p.stage_bytes;
                    fb += 8;
                    if (++slot == p.S) {
                        slot = 0;
                        ph ^= 1u;
                        st = base;
                        fb = full;
                    }
                }
            }
        }
        __syncwarp();
    } else if (warp == kMma) {
        // ------------------------------------------------------------ MMA issue
        // One thread walks the stages; descriptors and barriers advance with the slot.
        // In a pair the first CTA's thread issues for both.
        if (rank == 0 && elect_one()) {
        constexpr uint32_t kHi = (1024u >> 4) | (1u << 14) | (2u << 29);   // sw128_desc's upper word
        const uint32_t lo0 = ((base >> 4) & 0x3FFFu) | (1u << 16), lo_step = p.stage_bytes >> 4, lo_b = p.off_b >> 4;
        auto desc = [](uint32_t lo) { return ((uint64_t)kHi << 32) | lo; };
        Walk wk(work, worker);
        Seg sg;
        Ring rt, ra;
        int slot = 0;
        uint32_t ph = 0, fb = full, lo = lo0, sf = tmem + p.sf_col0;
        bool ok = true;
        Tile t;
        while (ok && wk.next(p, tl, pl, sg, t)) {
            const int nN = mma_n<SRC, CG>(t.rows);
            const uint32_t idesc = SRC == kGroupMx8    ? idesc_mx8(CG, nN, 0)
                                   : SRC == kGroupMxMx ? idesc_mx(CG, nN, 0)
                                                       : mma_idesc_bf16(CG * kTileN, nN);
            if (!wait_pair<CG>(acce + 8 * ra.i, ra.ph ^ 1u, p.timeout, abort_flag)) { ok = false; break; }
            tc_fence_after();
            const uint32_t acc = tmem + (uint32_t)ra.i * p.acc_w;
            uint32_t more = 0;   // 0: the tile's first MMA overwrites
            for (int kt = sg.kt0; kt < sg.kt1; kt++) {
                if (kRe && !wait_one(recon + 8 * rt.i, rt.ph, p.timeout, abort_flag)) { ok = false; break; }
                // (scales joined on chip come after everything else of the stage)
                const uint32_t ready = SRC == kGroupMx8 && CG == 1 && p.up ? fb + (mixed - full) : fb;
                if (!wait_one(ready, ph, p.timeout, abort_flag)) { ok = false; break; }
                tc_fence_after();
                if (kScaled) {
                    // scales of the stage, 4 columns per 512 bytes: weights, then rows
                    const uint32_t ss = lo + (p.off_s >> 4), sb = lo + lo_b - (p.sf_b_bytes >> 4);
                    const uint32_t sfb = sf + (SRC == kGroupMxMx ? 8u : 4u);
                    // a tile of 192 slots may start in the middle of a scale tile: two columns on
                    const uint32_t sfx = SRC == kGroupMxMx ? sfb + (uint32_t)(t.s0 % kMxTileRows) / 32u : sfb;
                    if (SRC == kGroupMxMx) {
                        const uint32_t nb = p.sf_b_bytes / kMxTileBytes;
#pragma unroll
                        for (uint32_t h = 0; h < 2; h++) {
                            tc_copy_scales<CG>(sf + 4u * h, ss + 32u * h);
                            tc_copy_scales<CG>(sfb + 4u * h * nb, sb + 32u * h);
                            if (nb > 1) tc_copy_scales<CG>(sfb + 4u * (h * nb + 1), sb + 64u + 32u * h);
                        }
#pragma unroll
                        for (uint32_t j = 0; j < 4; j++, more = 1)
                            tc_mma_mx(acc, desc(lo + 2u * j), desc(lo + lo_b + 2u * j), idesc + (j & 1u) * ((2u << 4) | (2u << 29)),
                                      sf + 4u * (j >> 1), sfx + 4u * nb * (j >> 1), more);
                    } else {
                        tc_copy_scales<CG>(sf, CG == 1 && p.up ? ss + 64u : ss);
                        tc_copy_scales<CG>(sfb, sb);
                        if (p.sf_b_bytes > 512u) tc_copy_scales<CG>(sfb + 4u, sb + 32u);
#pragma unroll
                        for (uint32_t j = 0; j < 4; j++, more = 1)
                            tc_mma_mx8<CG>(acc, desc(lo + 2u * j), desc(lo + lo_b + 2u * j), idesc + j * ((1u << 4) | (1u << 29)), sf, sfx,
                                       more);
                    }
                    sf += p.sf_slot;
                } else {
                    const uint32_t ta = tmem + p.a_col0 + (uint32_t)(KB / 2) * (uint32_t)rt.i;
#pragma unroll
                    for (uint32_t j = 0; j < 4; j++, more = 1) {
                        if (kRe)
                            tc_mma_tmem_a(acc, ta + 8u * j, desc(lo + lo_b + 2u * j), idesc, more);
                        else
                            tc_mma_bf16<CG>(acc, desc(lo + 2u * j), desc(lo + lo_b + 2u * j), idesc, more);
                    }
                }
                pair_commit<CG>(fb + 8 * kMaxS);   // empty
                if (kRe) {
                    tc_commit(tfree + 8 * rt.i);
                    rt.advance(p.T);
                }
                lo += lo_step;
                fb += 8;
                if (++slot == p.S) {
                    slot = 0;
                    ph ^= 1u;
                    lo = lo0;
                    fb = full;
                    sf = tmem + p.sf_col0;
                }
            }
            if (!ok) break;
            pair_commit<CG>(accf + 8 * ra.i);
            ra.advance(p.nacc);
        }
        // drain the tensor core before tensor memory is released
        pair_commit<CG>(fin);
        mbar_wait(fin, 0, p.timeout, nullptr);
        }
        __syncwarp();
    } else if (SRC == kGroupMx8 && CG == 1 && (warp == kMix || warp == kMix2)) {
        // ------------------------------------------------------------ scales of two weights
        // The tile's 128 rows are 64 of W and 64 of `up`, halves of a 128-row
        // scale tile each: lane l joins the 8 bytes of its rows l and l + 32 of
        // either into the 16 bytes that tensor memory takes for lane l.  (Pairs find
        // them joined in the workspace: what the second CTA's warps write would have
        // to be released to the first's MMAs at cluster scope, about 1600 cycles a
        // stage.)  A stage
        // costs a warp some 450 cycles of latency, so two share the slots (8 experts of
        // 14336 x 4096 twice, 16 rows: 96 us, 108 with one).
        if (p.up) {
            const int mine = warp == kMix ? 0 : 1;
            Walk wk(work, worker);
            Seg sg;
            Ring r;
            bool ok = true;
            Tile t;
            while (ok && wk.next(p, tl, pl, sg, t)) {
                for (int kt = sg.kt0; kt < sg.kt1; kt++, r.advance(p.S)) {
                    if (slot_warp(r.i) != mine) continue;
                    if (!mbar_wait(full + 8 * r.i, r.ph, p.timeout, abort_flag)) { ok = false; break; }
                    const uint32_t ss = base + (uint32_t)r.i * p.stage_bytes + p.off_s;
                    const uint32_t at = ss + (uint32_t)(lane * 16 + (t.n & 1) * 8);
                    const uint32_t to = ss + 1024u + (uint32_t)(lane * 16);
#pragma unroll
                    for (uint32_t i = 0; i < 2; i++) {
                        sts32(to + 4u * i, lds32(at + 4u * i));
                        sts32(to + 8u + 4u * i, lds32(at + 512u + 4u * i));
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(mixed + 8 * r.i);
                }
            }
        }
    } else if (kRe && warp >= kRebuild0) {
        // ------------------------------------------------------------ rebuild
        // Warp w owns tensor-memory lanes (weight rows) 32 (w % 4) ..; the two
        // warps of a quarter take one piece of 32 k each.
        const int quarter = warp & 3, pc = (warp - kRebuild0) >> 2;
        const int row = 32 * quarter + lane;
        Walk wk(work, worker);
        Seg sg;
        Ring r, rt;
        bool ok = true;
        Tile t;
        while (ok && wk.next(p, tl, pl, sg, t)) {
            // where this row's scale bytes are in the stage
            uint32_t so = p.off_s;
            int sq = quarter;
            if (p.up) {
                so += quarter >= 2 ? p.sf_a_bytes : 0;
                sq = (quarter & 1) + (t.n & 1) * 2;
            }
            so += (uint32_t)(lane * 16 + sq * 4);
            for (int kt = sg.kt0; kt < sg.kt1; kt++, r.advance(p.S), rt.advance(p.T)) {
                if (!mbar_wait(full + 8 * r.i, r.ph, p.timeout, abort_flag)) { ok = false; break; }
                if (!mbar_wait(tfree + 8 * rt.i, rt.ph ^ 1u, p.timeout, abort_flag)) { ok = false; break; }
                tc_fence_after();
                const uint32_t st = base + (uint32_t)r.i * p.stage_bytes;
                const uint4 c = lds128(st + sw32(row, pc));
                const uint32_t word = lds32(st + so);
                uint32_t out[16];
                rebuild32(c, (word >> (16 * (kt & 1) + 8 * pc)) & 255u, out);
                tmem_st16(tmem + p.a_col0 + (uint32_t)(KB / 2) * (uint32_t)rt.i + 16u * (uint32_t)pc + ((uint32_t)(32 * quarter) << 16),
                          out);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(recon + 8 * rt.i);
            }
        }
    } else if (warp < kEpiWarps) {
        // ------------------------------------------------------------ epilogue
        // Warps q and q + 4 share the tile's rows 32 q ..; of every 64 slots each
        // takes 32.
        const int quarter = warp & 3, set = warp >> 2;
        const int row = quarter * 32 + lane;
        const uint32_t trow = tmem + ((uint32_t)(quarter * 32) << 16);
        const uint32_t stg = base + p.stg_off + (uint32_t)warp * kWarpStage, xch = base + p.stg_off + kEpiWarps * kWarpStage;
        const size_t slot_f4 = (size_t)p.part_f4 * kTileN;   // float4s of a CTA's partial
        Walk wk(work, worker);
        Seg sg;
        Ring ra;
        Tile t;
        while (wk.next(p, tl, pl, sg, t)) {
            const int cols = (t.rows + 15) & ~15;
            const uint32_t lo = (uint32_t)(mma_n<SRC, CG>(t.rows) / 2);   // split rows: first lo column
            const bool publish = publishes(sg);
            // the tile's other ranges, in k order: workers worker + stride, ... up to `last`
            const int stride = (int)join_stride(pl), last = (int)last_joined(pl, sg, (uint32_t)worker);
            bool good = true;
            for (int b = worker + stride; good && b <= last; b += stride)
                good = wait_tag(p.flags + (size_t)(b * CG + rank) * kEpiWarps + warp, p.epoch, p.timeout, abort_flag);
            if (good) good = mbar_wait(accf + 8 * ra.i, ra.ph, p.timeout, abort_flag, 20000);
            if (any_of_epilogue(!good)) break;
            tc_fence_after();
            const uint32_t acc = trow + (uint32_t)ra.i * p.acc_w;
            // The accumulator is free once this warp has read its share.  Nothing was written that the MMAs which overwrite it
            // would read, so a relaxed arrival at cluster scope will do: it is the form that the PTX manual gives for a
            // tcgen05.ld before another thread's tcgen05.mma (wait::ld, fence::before_thread_sync, relaxed arrive; wait,
            // fence::after_thread_sync, mma).
            auto release = [&]() {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (CG == 2) arrive_at(in_first(acce + 8 * ra.i));
                    else mbar_arrive(acce + 8 * ra.i);
                }
            };
            // 16 slots of the accumulator (hi + lo of split rows)
            auto take = [&](int c, uint32_t (&v)[16]) {
                tmem_ld16(acc + (uint32_t)c, v);
                if (SRC == kGroupMx8) {
                    uint32_t l[16];
                    tmem_ld16(acc + lo + (uint32_t)c, l);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 16; i++) v[i] = __float_as_uint(__uint_as_float(v[i]) + __uint_as_float(l[i]));
                } else {
                    tmem_wait_ld();
                }
            };
            if (publish) {
                float4* dst = reinterpret_cast<float4*>(p.partial) + (size_t)(worker * CG + rank) * slot_f4 + row;
                for (int c = 0; c < cols; c += 16) {
                    if ((c >> 5 & 1) != set) continue;
                    uint32_t v[16];
                    take(c, v);
#pragma unroll
                    for (int i = 0; i < 4; i++)
                        __stcg(dst + (size_t)(c / 4 + i) * kTileN,
                               make_float4(__uint_as_float(v[4 * i]), __uint_as_float(v[4 * i + 1]),
                                           __uint_as_float(v[4 * i + 2]), __uint_as_float(v[4 * i + 3])));
                }
                release();   // (synchronises the warp: the tag's release covers every lane's stores)
                if (lane == 0)
                    asm volatile("st.release.gpu.global.u64 [%0], %1;" ::"l"(p.flags + (size_t)(worker * CG + rank) * kEpiWarps + warp),
                                 "l"(p.tag)
                                 : "memory");
            } else {
                // 16 slots of the finished sum: the accumulator plus the other ranges' partial sums, in k order
                // (two ranges' loads at a time)
                auto sum = [&](int c, uint32_t (&v)[16]) {
                    take(c, v);
                    for (int b = worker + stride; b <= last; b += 2 * stride) {
                        const float4* src = reinterpret_cast<const float4*>(p.partial) + (size_t)(b * CG + rank) * slot_f4 + row +
                                            (size_t)(c / 4) * kTileN;
                        const size_t next = b + stride <= last ? (size_t)(stride * CG) * slot_f4 : 0;
                        float4 x[4], y[4];
#pragma unroll
                        for (int i = 0; i < 4; i++) x[i] = __ldcg(src + (size_t)i * kTileN);
#pragma unroll
                        for (int i = 0; i < 4; i++) y[i] = __ldcg(src + next + (size_t)i * kTileN);
#pragma unroll
                        for (int i = 0; i < 4; i++) {
                            v[4 * i] = __float_as_uint(__uint_as_float(v[4 * i]) + x[i].x);
                            v[4 * i + 1] = __float_as_uint(__uint_as_float(v[4 * i + 1]) + x[i].y);
                            v[4 * i + 2] = __float_as_uint(__uint_as_float(v[4 * i + 2]) + x[i].z);
                            v[4 * i + 3] = __float_as_uint(__uint_as_float(v[4 * i + 3]) + x[i].w);
                        }
                        if (next) {
#pragma unroll
                            for (int i = 0; i < 4; i++) {
                                v[4 * i] = __float_as_uint(__uint_as_float(v[4 * i]) + y[i].x);
                                v[4 * i + 1] = __float_as_uint(__uint_as_float(v[4 * i + 1]) + y[i].y);
                                v[4 * i + 2] = __float_as_uint(__uint_as_float(v[4 * i + 2]) + y[i].z);
                                v[4 * i + 3] = __float_as_uint(__uint_as_float(v[4 * i + 3]) + y[i].w);
                            }
                        }
                    }
                };
                // first output of this warp: 32 rows of W, or of W and `up` each (warps w and w + 2)
                const int64_t nw = ((int64_t)t.n * CG + rank) * rows_a + 32 * (p.up ? quarter & 1 : quarter);
                if (!p.up) {
                    for (int c = 32 * set; c < cols; c += 64) {
                        uint32_t v[2][16];
                        sum(c, v[0]);
                        const bool two = c + 16 < cols;
                        if (two) sum(c + 16, v[1]);
                        if (c + 64 >= cols) release();
                        store32(p, v, two, t.s0 + c, t.rows - c, nw, lane, stg);
                    }
                    if (32 * set >= cols) release();
                } else {
                    // Quarter q holds rows of W, quarter q + 2 the same rows of `up`: of every 32 slots the first
                    // computes 16 and gets their `up` sums, the second the other 16 and gets their W sums.
                    const uint32_t mine = xch + (uint32_t)warp * 2048u + (uint32_t)lane * 4u;
                    const uint32_t theirs = xch + (uint32_t)(warp ^ 2) * 2048u + (uint32_t)lane * 4u;
                    const bool first = quarter < 2;
                    const int bar = kEpiBarId + 1 + (quarter & 1) + 2 * set;
                    for (int c0 = 32 * set; c0 < cols; c0 += 64) {
                        uint32_t keep[16], give[16];
                        const int ck = c0 + (first ? 0 : 16), cg = c0 + (first ? 16 : 0);
                        if (cg < cols) {
                            sum(cg, give);
#pragma unroll
                            for (int i = 0; i < 16; i++) sts32(mine + (uint32_t)(128 * i), give[i]);
                        }
                        if (ck < cols) sum(ck, keep);
                        if (c0 + 64 >= cols) release();
                        named_bar_sync(bar, 64);
                        if (ck < cols) {
                            const int valid = t.rows - ck;
                            uint32_t o[16];
#pragma unroll
                            for (int i = 0; i < 16; i++) o[i] = lds32(theirs + (uint32_t)(128 * i));
#pragma unroll
                            for (int i0 = 0; i0 < 16; i0 += 8) {
                                if (i0 >= valid) break;
#pragma unroll
                                for (int i = i0; i < i0 + 8; i++) {
                                    const float g = __uint_as_float(first ? keep[i] : o[i]), u = __uint_as_float(first ? o[i] : keep[i]);
                                    keep[i] = __float_as_uint(silu(g) * u);
                                }
                            }
                            store16(p, keep, t.s0 + ck, valid, nw, lane, stg);
                        }
                        if (c0 + 64 < cols) named_bar_sync(bar, 64);   // the sums have been read
                    }
                    if (32 * set >= cols) release();
                }
                // the tags are cleared for a replay of this call
                if (lane == 0)
                    for (int b = worker + stride; b <= last; b += stride) p.flags[(size_t)(b * CG + rank) * kEpiWarps + warp] = 0ull;
            }
            ra.advance(p.nacc);
        }
    }

    tc_fence_before();
    __syncthreads();
    // On expiry a role may have issued loads for a stage that the others did not come to; no barrier shows when these
    // have landed, so they are given a thousand times a load's latency.  (Nothing is issued any more.)
    if (*abort_flag)
        for (const uint64_t end = globaltimer() + kRestNs; globaltimer() < end;) {}
    // No CTA leaves while the other's MMAs or arrivals reach it: the commits' arrivals have been waited for (kProd), the
    // warps' are ordered by this barrier.
    if (CG == 2) cluster_sync();
    if (*abort_flag && threadIdx.x == 0) raise_status(UW_ERR_TIMEOUT);
    if (warp == kMma) {
        tc_fence_after();
        pair_dealloc<CG>(tmem, kTmemCols);
    }
}

template <int SRC, int CG>
__global__ void __launch_bounds__(SRC == kGroupMx8 && CG == 1 ? kThreadsMix : kThreadsPlain, 1)
    k_group(const __grid_constant__ Maps m, const GroupParams p) {
    group_body<SRC, CG>(m, p);
}

__global__ void __launch_bounds__(kThreadsRebuild, 1)
    k_group_rebuild(const __grid_constant__ Maps m, const GroupParams p) {
    group_body<kGroupMx, 1>(m, p);
}

// ---------------------------------------------------------------- rows before the product
struct PrepParams {
    const uint16_t* X;
    const int32_t* rows;      // NULL: slot s is row s
    const int32_t* offsets;
    int64_t x_rows, slots, K;
    int E, MG, kt, round, step;
    int steps;                // split rows: 512 k at a time of a warp's item
    uint32_t sf_bytes;        // scale bytes in front of a stage's rows
    int64_t chunk;
    uint8_t* out;
    const uint8_t* sw;        // scale tiles of two weights to be joined
    const uint8_t* su;
    uint8_t* joined;          // NULL: not wanted
    int row_tiles, k_tiles;   // of one matrix
};

constexpr int kPrepThreads = 256;
constexpr int kPrepK = 512;     // k of a warp's step: 16 a lane

// 16 values of a row as hi and lo, and the scale byte of their block of 32 (its
// other half is in the neighbouring lane).
struct Split16 {
    uint32_t hi[4], lo[4], sb;
};

// By fp32, whatever the values: tiny blocks, subnormals, NaN and infinities
// (which become NaN: e4m3 has no infinity).
// (By value: a reference would keep every result in local memory.)
__device__ __noinline__ Split16 split16_any(const uint4 a, const uint4 b) {
    Split16 q;
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    float v[16];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; i++) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
#pragma unroll
    for (int i = 0; i < 16; i++) {
        const uint32_t x = __float_as_uint(v[i]) & 0x7FFFFFFFu;
        if (x < 0x7F800000u) top = top > x ? top : x;
        else v[i] = __uint_as_float(0x7FC00000u);
    }
    const uint32_t other = __shfl_xor_sync(0xFFFFFFFFu, top, 1);
    top = top > other ? top : other;
    // scale 2^s puts the largest into [2^7, 2^8); its byte also has to hold s - 4
    const uint32_t ex = top >> 23;                        // floor(log2) + 127
    q.sb = ex > 11u ? ex - 7u : 4u;                       // s + 127
    const float inv = __uint_as_float((254u - q.sb) << 23);
#pragma unroll
    for (int i = 0; i < 4; i++) {
        uint32_t h2[2];
        float d[4];
#pragma unroll
        for (int j = 0; j < 4; j++) d[j] = v[4 * i + j] * inv;
        asm("{\n\t.reg .b16 x, y;\n\t"
            "cvt.rn.satfinite.e4m3x2.f32 x, %4, %3;\n\t"
            "cvt.rn.satfinite.e4m3x2.f32 y, %6, %5;\n\t"
            "mov.b32 %0, {x, y};\n\t"
            "cvt.rn.f16x2.e4m3x2 %1, x;\n\t"
            "cvt.rn.f16x2.e4m3x2 %2, y;\n\t}"
            : "=r"(q.hi[i]), "=r"(h2[0]), "=r"(h2[1])
            : "f"(d[0]), "f"(d[1]), "f"(d[2]), "f"(d[3]));
#pragma unroll
        for (int j = 0; j < 2; j++) {
            const __half2 h = *reinterpret_cast<const __half2*>(&h2[j]);
            d[2 * j] = (d[2 * j] - __low2float(h)) * 16.0f;
            d[2 * j + 1] = (d[2 * j + 1] - __high2float(h)) * 16.0f;
        }
        asm("{\n\t.reg .b16 x, y;\n\t"
            "cvt.rn.satfinite.e4m3x2.f32 x, %2, %1;\n\t"
            "cvt.rn.satfinite.e4m3x2.f32 y, %4, %3;\n\t"
            "mov.b32 %0, {x, y};\n\t}"
            : "=r"(q.lo[i])
            : "f"(d[0]), "f"(d[1]), "f"(d[2]), "f"(d[3]));
    }
    return q;
}

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
    uint32_t m;
    asm("max.u16x2 %0, %1, %2;" : "=r"(m) : "r"(a), "r"(b));
    return m;
}

// Blocks whose largest value is a normal number from 2^-104 on (or all zero):
// in pairs.  |x| 2^-s as an fp16 number v is the BF16 bits with the exponent
// field moved, (bits - ((s + 112) << 7)) << 3; what is below 2^-14 there (2^-21 of
// the block's largest) lands somewhere below 2^-14.  v 2^-8 has e4m3's exponent
// field and subnormal range in bits 13..10 and its mantissa below them, so
// hi is its upper bits, cut off; the rest, at most 4 significant bits
// where hi is normal, gives lo the same way, rounded.
__device__ __forceinline__ Split16 split16(const uint4 a, const uint4 b) {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; i++) m = max_u16x2(m, w[i] & 0x7FFF7FFFu);
    uint32_t top = (m & 0xFFFFu) > (m >> 16) ? m & 0xFFFFu : m >> 16;
    const uint32_t other = __shfl_xor_sync(0xFFFFFFFFu, top, 1);
    top = top > other ? top : other;
    const uint32_t ex = top >> 7;
    if (__any_sync(0xFFFFFFFFu, (ex < 23u && top) || ex == 255u)) return split16_any(a, b);
    Split16 q;
    q.sb = top ? ex - 7u : 16u;
    const uint32_t c = (q.sb - 15u) << 7, c2 = c | (c << 16);
    const __half2 down8 = __float2half2_rn(0x1p-8f), down4 = __float2half2_rn(0x1p-4f), n16 = __float2half2_rn(-16.0f);
#pragma unroll
    for (int i = 0; i < 4; i++) {
        uint32_t hi[2], lo[2];
#pragma unroll
        for (int j = 0; j < 2; j++) {
            const uint32_t t = (max_u16x2(w[2 * i + j] & 0x7FFF7FFFu, c2) - c2) << 3;
            const __half2 v = *reinterpret_cast<const __half2*>(&t), u = __hmul2(v, down8);
            const uint32_t ub = *reinterpret_cast<const uint32_t*>(&u), hb = ub & 0xFF80FF80u;
            const __half2 r = __hfma2(*reinterpret_cast<const __half2*>(&hb), n16, __hmul2(v, down4));   // 16 (v 2^-8 - hi 2^-8)
            hi[j] = ub << 1;
            lo[j] = (*reinterpret_cast<const uint32_t*>(&r) << 1) + 0x00800080u;
        }
        const uint32_t sign = prmt(w[2 * i], w[2 * i + 1], 0x7531u) & 0x80808080u;
        q.hi[i] = prmt(hi[0], hi[1], 0x7531u) | sign;
        q.lo[i] = prmt(lo[0], lo[1], 0x7531u) | sign;
    }
    return q;
}

// Scales of W and `up` for a pair of CTAs, each with 64 rows of either: of the
// 16 bytes that a half scale tile holds for lane l (rows l, l + 32, l + 64, l +
// 96) the first CTA takes the first 8 of W and of `up`, the second the last 8.
// Row ((expert, 64 weight rows), k step) of `joined` is 512 bytes.  A warp joins
// one scale tile of either weight at a time; bound by reading and writing one
// byte per 32 weights (11.5 MB of two 64 x 1408 x 2048 weights: 3 us of the split's 25).
__device__ __forceinline__ void join_scales(const PrepParams& p, const int32_t* count, uint32_t w0, uint32_t warps) {
    const int lane = threadIdx.x & 31;
    const uint32_t per = (uint32_t)(p.row_tiles * p.k_tiles), items = (uint32_t)p.E * per;   // (below 2^31: one CTA quantises a tile)
    for (uint32_t i = w0; i < items; i += warps) {
        const uint32_t e = i / per, t = i - e * per, rt = t / (uint32_t)p.k_tiles, kt = 2u * (t - rt * (uint32_t)p.k_tiles);
        if (!count[e]) continue;   // no tile reads them
        const uint4* w = reinterpret_cast<const uint4*>(p.sw + (int64_t)i * kMxTileBytes) + lane;
        const uint4* u = reinterpret_cast<const uint4*>(p.su + (int64_t)i * kMxTileBytes) + lane;
        const uint4 a[2] = {__ldg(w), __ldg(w + 32)}, b[2] = {__ldg(u), __ldg(u + 32)};
        uint4* out = reinterpret_cast<uint4*>(p.joined) + (2 * ((int64_t)e * p.row_tiles + rt) * p.kt + kt) * 32 + lane;
#pragma unroll
        for (int h = 0; h < 2; h++) {
            if (kt + h >= (uint32_t)p.kt) break;   // K an odd multiple of 128
            out[h * 32] = make_uint4(a[h].x, a[h].y, b[h].x, b[h].y);
            out[((int64_t)p.kt + h) * 32] = make_uint4(a[h].z, a[h].w, b[h].z, b[h].w);
        }
    }
}

// Rows of split tiles.  A warp takes `steps` (1 or 2) times 512 k of one slot
// at a time, 16 values a lane and step, two lanes a block of 32; slots are
// dealt out evenly whatever the groups are.  Row r of a tile of n (rounded up
// to 8, pairs 16) rows becomes row r (hi) and n + r (lo) of every stage's
// 128-byte swizzled rows; their scale bytes lie in front as tcgen05.cp reads
// them.  Reads and writes stay in L2 mostly (a row is read once for each of its
// slots); bound by instructions (12288 slots of 2048: 22 us, 2.3 TB/s each way,
// 25 us with the joined scales of 64 experts of 1408 x 2048; 4480 rows of 4096: 16 us).
__global__ void __launch_bounds__(kPrepThreads, 4) k_group_split(const PrepParams p) {
    extern __shared__ int32_t tab[];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    int32_t* cum = tab;
    int32_t* begin = cum + p.E + 1;
    int32_t* count = begin + p.E;
    const int lane = threadIdx.x & 31;
    list_tiles(p.offsets, p.E, p.slots, p.MG, 1, cum, begin, count);
    if (cum[p.E] == 0) return;
    uint32_t* each = reinterpret_cast<uint32_t*>(count + p.E);   // slots of an expert's tiles
    for (int e = threadIdx.x; e < p.E; e += kPrepThreads) each[e] = count[e] ? (uint32_t)tile_slots(count[e], p.MG, p.step) : 1u;
    __syncthreads();
    const uint32_t s_first = (uint32_t)begin[0], s_end = (uint32_t)(begin[p.E - 1] + count[p.E - 1]);
    const uint32_t segs = (uint32_t)((p.K + kPrepK * p.steps - 1) / (kPrepK * p.steps));
    const uint32_t warps = gridDim.x * (kPrepThreads / 32), ds = warps / segs, dseg = warps % segs;
    const uint32_t w0 = blockIdx.x * (kPrepThreads / 32) + (threadIdx.x >> 5);
    const int unit = lane & 7;   // 16-byte unit of the stage's row
    bool wrong = false;
    if (p.joined) join_scales(p, count, w0, warps);
    uint32_t seg = w0 % segs;
    for (uint32_t s = s_first + w0 / segs; s < s_end;) {
        int64_t row = s;
        if (p.rows) {
            const int32_t v = __ldg(p.rows + s);
            const bool ok = v >= 0 && v < p.x_rows;
            wrong |= !ok;
            row = ok ? v : 0;
        }
        const int k0 = (int)seg * kPrepK * p.steps + 16 * lane;
        uint4 in[2][2] = {};
#pragma unroll
        for (int i = 0; i < 2; i++)
            if (i < p.steps && k0 + i * kPrepK < p.K) {   // K is a multiple of 128: the 8 lanes of a stage agree
                const uint4* src = reinterpret_cast<const uint4*>(p.X + row * p.K + k0 + i * kPrepK);
                in[i][0] = __ldg(src);
                in[i][1] = __ldg(src + 1);
            }
        // meanwhile: the slot's tile (the last expert that begins at it or before has it)
        int e = 0;
        for (int hi = p.E; hi - e > 1;) {
            const int mid = (e + hi) >> 1;
            if ((uint32_t)begin[mid] <= s) e = mid; else hi = mid;
        }
        const uint32_t n = each[e], in_group = s - (uint32_t)begin[e], m = in_group / n;
        const int rh = (int)(in_group - m * n), left = count[e] - (int)(m * n), nrows = left < (int)n ? left : (int)n;
        const int rl = ((nrows + p.round - 1) & ~(p.round - 1)) + rh;   // as mma_n
        uint8_t* tile = p.out + (int64_t)(cum[e] + (int)m) * p.kt * p.chunk;
        auto at = [](int r) { return (r >> 7) * 512 + (r & 31) * 16 + ((r >> 5) & 3) * 4; };
        const int sh = at(rh), sl = at(rl);
        const uint32_t bh = p.sf_bytes + rh * 128 + ((unit ^ (rh & 7)) << 4), bl = p.sf_bytes + rl * 128 + ((unit ^ (rl & 7)) << 4);
#pragma unroll
        for (int i = 0; i < 2; i++) {
            if (i >= p.steps) break;
            const Split16 q = split16(in[i][0], in[i][1]);
            // the four scale bytes of the stage's row, in every lane of its eight
            uint32_t sw = q.sb << (8 * (unit >> 1));
            sw |= __shfl_xor_sync(0xFFFFFFFFu, sw, 2);
            sw |= __shfl_xor_sync(0xFFFFFFFFu, sw, 4);
            const int k = k0 + i * kPrepK;
            if (k < p.K) {
                uint8_t* out = tile + (int64_t)(k >> 7) * p.chunk;
                *reinterpret_cast<uint4*>(out + bh) = make_uint4(q.hi[0], q.hi[1], q.hi[2], q.hi[3]);
                *reinterpret_cast<uint4*>(out + bl) = make_uint4(q.lo[0], q.lo[1], q.lo[2], q.lo[3]);
                if (unit == 0) *reinterpret_cast<uint32_t*>(out + sh) = sw;
                if (unit == 1) *reinterpret_cast<uint32_t*>(out + sl) = sw - 0x04040404u;
            }
        }
        s += ds;
        seg += dseg;
        if (seg >= segs) {
            seg -= segs;
            s++;
        }
    }
    if (wrong) raise_status(UW_ERR_DEVICE);
}

// Gathered copy: Xs[s] = X[rows[s]] for the slots of the groups, 16 bytes a
// thread and step, four in flight.  Bound by reading and writing a row a slot.
__global__ void __launch_bounds__(kPrepThreads) k_group_gather(const PrepParams p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int64_t first = p.offsets ? p.offsets[0] : 0, end = p.offsets ? p.offsets[p.E] : p.slots;
    const int per = (int)(p.K / 8);   // 16-byte pieces of a row
    const int64_t stop = end < p.slots ? end : p.slots;
    for (int64_t s = (first > 0 ? first : 0) + blockIdx.x; s < stop; s += gridDim.x) {
        const int32_t v = p.rows[s];
        const bool in = v >= 0 && v < p.x_rows;
        if (!in && threadIdx.x == 0) raise_status(UW_ERR_DEVICE);
        const uint4* src = reinterpret_cast<const uint4*>(p.X + (in ? (int64_t)v : 0) * p.K);
        uint4* dst = reinterpret_cast<uint4*>(p.out) + s * per;
#pragma unroll 4
        for (int i = threadIdx.x; i < per; i += kPrepThreads) dst[i] = __ldg(src + i);
    }
}

// Slots of a tile: twice the mean group (groups are uneven), a power of two
// from 16 up.  At most 256; 112 split rows (two accumulators and the scales
// fit tensor memory).  Block-scaled products take 128 or 192: two accumulators
// and the scales fit, and tiles start at half a scale tile at worst.
int pick_tile_slots(int src, int64_t slots, int E) {
    const int64_t groups = E < slots ? E : slots;
    const int64_t mean = (slots + groups - 1) / groups;
    const int64_t want = E == 1 ? mean : 2 * mean;
    int mg = src == kGroupMxMx ? 128 : 16;
    while (mg < 256 && mg < want) mg *= 2;
    if (src == kGroupMx8 && mg > 64) mg = 112;
    if (src == kGroupMxMx && mg > 128) mg = 192;
    return mg;
}

// Pairs of CTAs where tiles are large: a pair reads half of X per CTA, which
// brings the bytes an SM has to take in below what L2 delivers (about 65 a
// cycle) per MMA cycle.
bool pick_pair(int src, int mg) { return src != kGroupMx && mg > 64; }

// How tiles that fill no round are cut.  Contiguous ranges keep every SM
// reading to the end, which small tiles (bound by reading weights) need.
// With pairs the workers of a round share weight and slot tiles in L2 because
// they walk k together; ranges that start anywhere lose that (8 experts of
// 1024 rows, 4096 x 14336 in BF16: 728 us with ranges, 660 with parts).
bool pick_parts(int CG) { return CG == 2; }

constexpr size_t al256(size_t x) { return (x + 255) & ~size_t(255); }

// How a call is cut up; the workspace holds partial sums, their tags, the
// prepared rows and the joined scales.
struct Shape {
    int MG = 0, KB = 0, kt = 0, n_tiles = 0;
    int CG = 1;               // CTAs of a worker
    int64_t m_tiles = 0;      // slot tiles at most
    bool gather = false;      // a gathered copy of BF16 rows
    uint32_t sf_b = 0;        // scale bytes of a stage's rows
    int64_t chunk = 0;        // split rows: bytes of a stage
    size_t partial = 0, flags = 0, prep = 0, joined = 0;
    size_t bytes() const { return partial + flags + prep + joined; }
};

Shape shape_of(int src, int64_t slots, int E, int64_t N, int64_t K, bool up, bool rows) {
    Shape h;
    const int P = num_sms();
    h.MG = pick_tile_slots(src, slots, E);
    h.KB = stage_k(src);
    h.kt = (int)((K + h.KB - 1) / h.KB);
    h.CG = pick_pair(src, h.MG) ? 2 : 1;
    const int rows_a = h.CG * (up ? kTileN / 2 : kTileN);
    h.n_tiles = (int)((N + rows_a - 1) / rows_a);
    h.m_tiles = slots / h.MG + (E < slots ? E : slots);
    h.partial = (size_t)P * h.MG * kTileN * 4;
    h.flags = al256((size_t)P * kEpiWarps * 8);
    if (src == kGroupMx8) {
        h.sf_b = 512u * (uint32_t)((2 * h.MG + 127) / 128);
        h.chunk = (int64_t)h.sf_b + 2 * h.MG * 128;
        h.prep = al256((size_t)h.m_tiles * h.kt * h.chunk);
        if (up && h.CG == 2) h.joined = (size_t)E * 2 * (size_t)mx_row_tiles(N) * (size_t)h.kt * (kMxTileBytes / 2);
    } else if (src == kGroupMxMx) {
        h.sf_b = (uint32_t)mx_row_tiles(h.MG) * kMxTileBytes;
    } else if (rows && h.MG > 32) {
        h.gather = true;
        h.prep = al256((size_t)slots * (size_t)K * 2);
    }
    return h;
}

// Test hook (UW_DEBUG_SKIP_TAGS=1, read once): cut tiles' partial sums are
// published under a tag that nobody waits for, so that the wait for them runs
// out.
bool skip_tags() {
    static const bool skip = [] {
        const char* e = getenv("UW_DEBUG_SKIP_TAGS");
        return e && e[0] == '1';
    }();
    return skip;
}

// The unpacking TMA load takes rows of whole 128 codes.
int resolve(int src, int64_t K) { return src == kGroupMx && K % 128 == 0 ? kGroupMx8 : src; }

template <typename K, typename... A>
cudaError_t launch_after(K kern, dim3 grid, int cluster, int threads, size_t smem, cudaStream_t s, const A&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args...);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

size_t group_ws_bytes(int src, int64_t slots, int E, int64_t N, int64_t K, bool up, bool rows) {
    return slots <= 0 ? 0 : shape_of(resolve(src, K), slots, E, N, K, up, rows).bytes();
}

cudaError_t launch_group(const GroupGemm& a, cudaStream_t s, uw_status* st) {
    *st = UW_OK;
    if (a.slots == 0) return cudaSuccess;
    const int src = resolve(a.src, a.K);
    const Shape h = shape_of(src, a.slots, a.E, a.N, a.K, a.up != nullptr, a.rows != nullptr);
    const int MG = h.MG, P = num_sms();
    const int64_t max_tiles = h.m_tiles * (int64_t)h.n_tiles;
    // 31-bit tiles; (k steps of two rounds) * CTAs in 32 bits
    if (max_tiles > 0x7FFFFFFF || 2 * (int64_t)P * P * h.kt >= (int64_t(1) << 32)) { *st = UW_ERR_SHAPE; return cudaSuccess; }
    if (!a.ws || a.ws_bytes < h.bytes()) { *st = UW_ERR_WORKSPACE; return cudaSuccess; }
    uint8_t* prep = (uint8_t*)a.ws + h.partial + h.flags;
    GroupParams p{};
    p.x_rows = a.x_rows;
    p.slots = a.slots;
    p.N = a.N;
    p.rows = src == kGroupMx8 || h.gather ? nullptr : a.rows;
    p.offsets = a.offsets;
    p.E = a.E;
    p.kt = h.kt;
    p.MG = MG;
    const int CG = h.CG;
    // divides MG / CG: boxes never pass the rows set aside.  (Split rows: one box whatever the tile holds; seven of
    // 16 rows cost the producer more than the bytes: 4480 x 8192 x 4096 248 us against 219.)
    p.box = src == kGroupMx8 ? MG : MG / CG % 64 ? MG / CG : 64;
    p.up = a.up ? 1 : 0;
    p.n_tiles = h.n_tiles;
    p.out_f32 = a.out_f32;
    p.y_vec = a.N % 8 == 0;
    p.Y = a.Y;
    p.sw = a.w_scales;
    p.su = a.up_scales;
    p.w_row_tiles = mx_row_tiles(a.N);
    p.k_tiles = (int)mx_k_tiles(a.K);
    p.early = src == kGroupMx8 || h.gather;
    p.parts = pick_parts(CG);
    // what the MMA's N rounds a tile to; half a scale tile for 4-bit rows
    p.step = src == kGroupMx8 ? 8 * CG : src == kGroupMxMx ? 64 : 16 * CG;
    p.prep = prep;
    p.prep_chunk = h.chunk;
    p.part_f4 = MG / 4;
    p.partial = (float*)a.ws;
    p.flags = (unsigned long long*)((uint8_t*)a.ws + h.partial);
    p.epoch = gemm_next_epoch();
    p.tag = skip_tags() ? ~0ull : p.epoch;   // (an epoch has 48 bits)
    p.timeout = timeout_ns();

    // stage: weight rows, their scales, the rows' scales, X (swizzled tiles 1024-byte aligned)
    auto al1k = [](uint32_t x) { return (x + 1023u) & ~1023u; };
    p.off_s = kTileN * (src == kGroupMx ? 32u : 128u);
    p.sf_a_bytes = src == kGroupBf16 ? 0 : src == kGroupMxMx ? kMxTileBytes : kMxTileBytes / 2;
    p.sf_b_bytes = h.sf_b;
    // (with `up`, split rows and a single CTA: a third part for the joined scales of both weights; pairs load them joined)
    p.off_b = al1k(p.off_s + p.sf_a_bytes * (p.up && CG == 1 ? (src == kGroupMx8 ? 3 : 2) : 1) + p.sf_b_bytes);
    p.stage_bytes = p.off_b + (uint32_t)(MG * 128 * (src == kGroupMx8 ? 2 : 1) / CG);
    const uint32_t ctrl = 1024, tab = (uint32_t)(3 * a.E + 1) * 4;
    const uint32_t epi = kEpiWarps * kWarpStage + (p.up ? kExchange : 0);
    const uint32_t tab16 = (tab + 15u) & ~15u, fixed = 1024 + ctrl + epi + tab16 + kListed * (uint32_t)sizeof(Work);
    // tensor memory: accumulators, then rebuilt-A slots (32 columns) or scale columns
    p.acc_w = (uint32_t)(src == kGroupMx8 ? 2 * MG : MG);
    p.sf_slot = src == kGroupMxMx ? 8u + 8u * (uint32_t)mx_row_tiles(MG) : src == kGroupMx8 ? 4u + h.sf_b / 128u : 0u;
    p.nacc = src == kGroupMx && MG > 128 ? 1 : 2;   // (rebuilt-A slots take half of tensor memory)
    const uint32_t acc_cols = (uint32_t)p.nacc * p.acc_w;
    int S = (int)((227 * 1024 - fixed) / p.stage_bytes);
    if (S > kMaxS) S = kMaxS;
    if (p.sf_slot && S > (int)((kTmemCols - acc_cols) / p.sf_slot)) S = (int)((kTmemCols - acc_cols) / p.sf_slot);
    if (src == kGroupMx) {
        p.T = (int)((kTmemCols - acc_cols) / 32u);
        if (p.T > kMaxT) p.T = kMaxT;
    }
    if (S < 2 || (src == kGroupMx && p.T < 2)) { *st = UW_ERR_UNSUPPORTED; return cudaSuccess; }
    p.S = S;
    p.a_col0 = p.sf_col0 = acc_cols;
    p.ctrl_off = (uint32_t)S * p.stage_bytes;
    p.stg_off = p.ctrl_off + ctrl;
    p.tab_off = p.stg_off + epi;
    p.work_off = p.tab_off + tab16;
    // One CTA per SM: each takes all of its tensor memory, and two calls on two streams whose CTAs wait for each other's
    // tensor memory and for their own grid's partial sums could stand still.
    const size_t one_per_sm = 116 * 1024, used = (size_t)S * p.stage_bytes + fixed, smem = used > one_per_sm ? used : one_per_sm;

    Maps m{};
    bool ok = true;
    const uint64_t wrows = (uint64_t)a.E * (uint64_t)a.N;
    if (src == kGroupMxMx)
        ok = make_map_2d(&m.x, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, a.X, a.K / 2, a.x_rows, a.K / 2, 128, p.box,
                         CU_TENSOR_MAP_SWIZZLE_128B);
    else if (src != kGroupMx8)
        ok = make_map_2d(&m.x, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, h.gather ? (const void*)prep : a.X, a.K,
                         h.gather ? a.slots : a.x_rows, a.K * 2, 64, p.rows ? 1 : p.box, CU_TENSOR_MAP_SWIZZLE_128B);
    else if (CG == 2)   // prepared rows: 128 bytes each, swizzled already
        ok = make_map_2d(&m.x, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, prep, 128, h.prep / 128, 128, 128, p.box, CU_TENSOR_MAP_SWIZZLE_NONE) &&
             make_map_2d(&m.sx, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, prep, 128, h.prep / 128, 128, 128, h.sf_b / 128,
                         CU_TENSOR_MAP_SWIZZLE_NONE);
    const uint32_t halves = src == kGroupMxMx ? 2 : 1;   // half scale tiles of a stage
    if (src == kGroupMxMx && CG == 2)
        ok = ok && make_map_2d(&m.sx, CU_TENSOR_MAP_DATA_TYPE_UINT32, 4, a.x_scales, 128,
                               2 * (uint64_t)mx_row_tiles(a.x_rows) * p.k_tiles, 512, 128, halves, CU_TENSOR_MAP_SWIZZLE_NONE);
    for (int i = 0; i < (a.up ? 2 : 1); i++) {
        const void* w = i ? a.up : a.W;
        CUtensorMap* mw = i ? &m.u : &m.w;
        if (src == kGroupBf16)
            ok = ok && make_map_2d(mw, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, w, a.K, wrows, a.K * 2, 64, kTileN / 2,
                                   CU_TENSOR_MAP_SWIZZLE_128B);
        else if (src == kGroupMx8)   // 16 packed codes -> 16 bytes of shared memory
            ok = ok && make_map_2d(mw, CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B, 1, w, a.K, wrows, a.K / 2, 128, kTileN / 2,
                                   CU_TENSOR_MAP_SWIZZLE_128B);
        else
            ok = ok && make_map_2d(mw, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, w, a.K / 2, wrows, a.K / 2, src == kGroupMx ? 32 : 128,
                                   kTileN / 2, src == kGroupMx ? CU_TENSOR_MAP_SWIZZLE_32B : CU_TENSOR_MAP_SWIZZLE_128B);
    }
    uint8_t* joined = h.joined ? prep + h.prep : nullptr;
    if (joined)
        ok = ok && make_map_2d(&m.sw, CU_TENSOR_MAP_DATA_TYPE_UINT32, 4, joined, 128, h.joined / 512, 512, 128, 1, CU_TENSOR_MAP_SWIZZLE_NONE);
    else if (CG == 2 && src != kGroupBf16)
        ok = ok && make_map_2d(&m.sw, CU_TENSOR_MAP_DATA_TYPE_UINT32, 4, a.w_scales, 128, 2 * (uint64_t)a.E * p.w_row_tiles * p.k_tiles,
                               512, 128, halves, CU_TENSOR_MAP_SWIZZLE_NONE);
    if (!ok) { *st = UW_ERR_CUDA; return cudaSuccess; }

    void (*kern)(const Maps, const GroupParams) =
        src == kGroupBf16   ? (CG == 2 ? k_group<kGroupBf16, 2> : k_group<kGroupBf16, 1>)
        : src == kGroupMxMx ? k_group<kGroupMxMx, 2>
        : src == kGroupMx8  ? (CG == 2 ? k_group<kGroupMx8, 2> : k_group<kGroupMx8, 1>)
                            : k_group_rebuild;
    cudaError_t e = set_smem_attr((const void*)kern, (int)smem);
    if (e != cudaSuccess) return e;

    if (p.early) {
        PrepParams q{};
        q.X = (const uint16_t*)a.X;
        q.rows = a.rows;
        q.offsets = a.offsets;
        q.x_rows = a.x_rows;
        q.slots = a.slots;
        q.K = a.K;
        q.E = a.E;
        q.MG = MG;
        q.kt = h.kt;
        q.round = 8 * CG;
        q.step = p.step;
        q.sf_bytes = h.sf_b;
        q.chunk = h.chunk;
        q.out = prep;
        if (src == kGroupMx8) {
            // warps take two steps at a time where that leaves none idle
            const int64_t one = a.slots * ((a.K + kPrepK - 1) / kPrepK), most = 4 * (int64_t)P;
            q.steps = one > 2 * most * (kPrepThreads / 32) ? 2 : 1;
            q.sw = a.w_scales;
            q.su = a.up_scales;
            q.joined = joined;
            q.row_tiles = (int)p.w_row_tiles;
            q.k_tiles = p.k_tiles;
            const int64_t items = joined ? a.E * p.w_row_tiles * p.k_tiles : 0;
            const int64_t ctas = ((one / q.steps > items ? one / q.steps : items) + kPrepThreads / 32 - 1) / (kPrepThreads / 32);
            e = launch_after(k_group_split, dim3((unsigned)(ctas < most ? ctas : most)), 1, kPrepThreads, tab + (size_t)a.E * 4, s, q);
        } else {
            e = launch_after(k_group_gather, dim3((unsigned)(a.slots < 8 * P ? a.slots : 8 * P)), 1, kPrepThreads, 0, s, q);
        }
        if (e != cudaSuccess) return e;
    }
    const int64_t workers = max_tiles * h.kt < P / CG ? max_tiles * h.kt : P / CG;
    return launch_after(kern, dim3((unsigned)(workers * CG)), CG,
                        src == kGroupMx ? kThreadsRebuild : src == kGroupMx8 && CG == 1 && p.up ? kThreadsMix : kThreadsPlain, smem, s, m, p);
}

}  // namespace uw
