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
//   * one persistent CTA per SM.  All full rounds of whole tiles but the last
//     are dealt out one tile a CTA; the rest is cut into equal k ranges, one
//     contiguous range a CTA, so every SM reads until the end.  The CTA with a
//     cut tile's first k steps reaches it last and adds the others' fp32
//     partial rows in k order (from the workspace; deterministic);
//   * warp roles: 0-3 epilogue, 4 TMA producer, 5 MMA issue, and for 4-bit
//     weights with BF16 rows 6-21 rebuild (codes -> BF16 in tensor memory, the
//     MMA's A operand).  Rows are gathered by the TMA (four row indices a
//     request);
//   * MXFP4 with MXFP4 rows: block-scaled MMA, the scale bytes go from shared
//     to tensor memory (tcgen05.cp) in the order the format stores them;
//   * every wait is bounded; on expiry the CTA raises UW_ERR_TIMEOUT, drains
//     its own copies and MMAs, frees tensor memory and returns.
#include "uw_device.cuh"
#include "uw_internal.h"

namespace uw {

int group_status_take() { return unit_status_take(); }

namespace {

constexpr int kTileN = 128;            // weight rows of a tile
constexpr int kProd = 4, kMma = 5, kRebuild0 = 6, kRebuildWarps = 16;
constexpr int kThreadsPlain = 6 * 32;
constexpr int kThreadsRebuild = (kRebuild0 + kRebuildWarps) * 32;
constexpr int kMaxS = 12;              // stages
constexpr int kMaxT = 8;               // rebuilt-A slots in tensor memory
constexpr int kBand = 16;              // slot tiles of a band
constexpr int kEpiBarId = 1;
constexpr int kChunk = 32;             // slots the epilogue moves at a time
constexpr uint32_t kStage32 = kChunk * kTileN * 4;   // epilogue staging: fp32 [32 slots][128 outputs]
constexpr uint32_t kTmemCols = 512;

struct GroupParams {
    int64_t x_rows, slots, N;
    const int32_t* rows;
    const int32_t* offsets;
    int E, kt, MG, box, n_tiles, up, out_f32, y_vec;
    int S, T, nacc;
    uint32_t stage_bytes, off_s, off_b;     // codes (or BF16 weights) at 0, scale bytes, X
    uint32_t sf_a_bytes, sf_b_bytes;        // scale bytes of a stage: weights (one matrix), X
    uint32_t a_col0, sf_col0;
    uint32_t ctrl_off, stg_off, tab_off;
    const uint8_t* sw;                      // scale tiles of W, up, X
    const uint8_t* su;
    const uint8_t* sx;
    int64_t w_row_tiles;                    // scale row tiles of one matrix
    int k_tiles;                            // scale tiles along k
    void* Y;
    float* partial;                         // [CTAs][MG/4][128] float4
    unsigned long long* flags;              // [CTAs][4]: call tag once a warp's partial rows are out
    unsigned long long epoch;
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

// The tile list as every role sees it (shared memory) and a CTA's share of it.
struct Plan {
    const int32_t* cum;      // [E + 1] tiles before each expert
    const int32_t* begin;    // [E] first slot
    const int32_t* count;    // [E] slots
    int64_t tiles, whole;    // tiles; tiles dealt out whole (the first ones)
    int64_t units;           // k steps of the cut tiles
    int ps;                  // CTAs that share them
};

struct Seg {
    int64_t tile;
    int kt0, kt1;
};

struct Tile {
    int e, n, rows;          // expert, weight tile, slots of the tile
    int64_t s0;              // first slot
};

// Units of CTA b's range start here; owner of a unit.
__device__ __forceinline__ int64_t unit_begin(int64_t b, const Plan& pl) { return b * pl.units / pl.ps; }
__device__ __forceinline__ int unit_owner(int64_t u, const Plan& pl) { return (int)(((u + 1) * pl.ps - 1) / pl.units); }

// A CTA's segments: its range of the cut tiles, then its whole tiles.
struct Walk {
    int64_t u, ue, t;
    __device__ __forceinline__ Walk(const Plan& pl, int b) {
        u = ue = 0;
        if (b < pl.ps) {
            u = unit_begin(b, pl);
            ue = unit_begin(b + 1, pl);
        }
        t = b;
    }
    __device__ __forceinline__ bool next(const Plan& pl, int kt, Seg& s) {
        if (u < ue) {
            s.tile = pl.whole + u / kt;
            s.kt0 = (int)(u % kt);
            const int64_t left = ue - u;
            s.kt1 = left < kt - s.kt0 ? s.kt0 + (int)left : kt;
            u += s.kt1 - s.kt0;
            return true;
        }
        if (t < pl.whole) {
            s.tile = t;
            s.kt0 = 0;
            s.kt1 = kt;
            t += gridDim.x;
            return true;
        }
        return false;
    }
};

__device__ __forceinline__ Tile locate(const GroupParams& p, const Plan& pl, int64_t tile) {
    int lo = 0, hi = p.E;   // last expert with cum[e] <= tile (experts without tiles are passed over)
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (pl.cum[mid] <= tile) lo = mid; else hi = mid;
    }
    const int c = pl.count[lo];
    const int mt = (c + p.MG - 1) / p.MG;
    int l = (int)(tile - pl.cum[lo]);
    const int band = l / (kBand * p.n_tiles);
    l -= band * kBand * p.n_tiles;
    const int nb = mt - band * kBand < kBand ? mt - band * kBand : kBand;
    Tile t;
    t.e = lo;
    t.n = l / nb;
    const int m = band * kBand + l % nb;
    t.s0 = (int64_t)pl.begin[lo] + (int64_t)m * p.MG;
    t.rows = c - m * p.MG < p.MG ? c - m * p.MG : p.MG;
    return t;
}

__device__ __forceinline__ uint16_t bf(float f) {
    const __nv_bfloat16 h = __float2bfloat16_rn(f);
    return *reinterpret_cast<const uint16_t*>(&h);
}
__device__ __forceinline__ uint32_t bf2(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ bool any_of_epilogue(bool pred) {
    uint32_t res;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "bar.red.or.pred q, %2, %3, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(res)
        : "r"((uint32_t)pred), "n"(kEpiBarId), "n"(4 * 32)
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

// 512 bytes of scales (32 rows x 16 bytes) -> 4 columns of tensor memory, in
// every quarter of the lanes.
__device__ __forceinline__ void tc_copy_scales(uint32_t tmem, uint32_t smem) {
    // rows of 16 bytes in 8-row groups of 128 bytes, no swizzle
    uint64_t d = (uint64_t)((smem >> 4) & 0x3FFFu);
    d |= (uint64_t)(128u >> 4) << 32;
    d |= (uint64_t)1u << 46;
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(d) : "memory");
}

// D (+)= A * B^T with e2m1 operands and one e8m0 scale per 32 k (K = 64).
__device__ __forceinline__ void tc_mma_mx(uint32_t d_tmem, uint64_t ad, uint64_t bd, uint32_t idesc, uint32_t sfa,
                                          uint32_t sfb, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d_tmem),
        "l"(ad), "l"(bd), "r"(idesc), "r"(sfa), "r"(sfb), "r"(acc)
        : "memory");
}

// Instruction descriptor of kind::mxf4: both operands e2m1, scales e8m0, both
// K-major, M = 128; `id` (0 or 2) picks the scale bytes' half word.
__device__ __forceinline__ uint32_t idesc_mx(int N, uint32_t id) {
    return (id << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | (1u << 23) | (1u << 27) | (id << 29);
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

__device__ __forceinline__ uint32_t swizzled(int row_bytes, int r, int c) {
    return row_bytes == 128  ? r * 128 + ((c ^ (r & 7)) << 4)
           : row_bytes == 64 ? r * 64 + ((c ^ ((r >> 1) & 3)) << 4)
                             : r * 32 + ((c ^ ((r >> 2) & 1)) << 4);
}

// SRC: kGroupBf16 (KB = 64 k a stage), kGroupMx (64, 128 or 256), kGroupMxMx (256).
template <int SRC, int KB>
__device__ __forceinline__ void group_body(const CUtensorMap& tm_x, const CUtensorMap& tm_w, const CUtensorMap& tm_u,
                                           const GroupParams& p) {
    constexpr bool kMx = SRC != kGroupBf16;
    constexpr bool kRe = SRC == kGroupMx;
    constexpr int kARow = SRC == kGroupBf16 ? 128 : KB / 2;          // bytes of a weight row in a stage
    constexpr int kHalves = SRC == kGroupMxMx ? 1 : KB / 64;         // 128-byte slabs of X
    constexpr int kGroups = KB == 64 ? 2 : 1;                        // rebuild groups (alternate stages)
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    uint8_t* smem = smem_raw + (base - smem_u32(smem_raw));
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + p.ctrl_off);
    const uint32_t full = smem_u32(bars), empty = full + 8 * kMaxS, recon = empty + 8 * kMaxS, tfree = recon + 8 * kMaxT;
    const uint32_t accf = tfree + 8 * kMaxT, acce = accf + 16, fin = acce + 16;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * kMaxS + 2 * kMaxT + 5);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    int32_t* cum = reinterpret_cast<int32_t*>(smem + p.tab_off);
    int32_t* begin = cum + p.E + 1;
    int32_t* count = begin + p.E;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < p.S; s++) {
            mbar_init(full + 8 * s, 1);
            mbar_init(empty + 8 * s, 1);
        }
        for (int t = 0; t < p.T; t++) {
            mbar_init(recon + 8 * t, kRebuildWarps / kGroups);
            mbar_init(tfree + 8 * t, 1);
        }
        for (int a = 0; a < 2; a++) {
            mbar_init(accf + 8 * a, 1);
            mbar_init(acce + 8 * a, 4);
        }
        mbar_init(fin, 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == kMma) {
        tmem_alloc(smem_u32(tmem_slot), kTmemCols);
        tmem_relinquish();
    }
    if (warp == kProd && lane == 0) {
        tma_prefetch_desc(&tm_x);
        tma_prefetch_desc(&tm_w);
        tma_prefetch_desc(&tm_u);
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (warp == 0) {
        // the tile list: 32 runs of experts, one a lane
        const int each = (p.E + 31) / 32, lo = lane * each < p.E ? lane * each : p.E, hi = lo + each < p.E ? lo + each : p.E;
        int sum = 0;
        bool bad = false;
        for (int e = lo; e < hi; e++) {
            int64_t b = 0, n = p.slots;
            if (p.offsets) {
                const int64_t o0 = p.offsets[e], o1 = p.offsets[e + 1];
                bad |= o0 < 0 || o1 < o0 || o1 > p.slots;
                b = o0 < 0 ? 0 : o0 > p.slots ? p.slots : o0;
                n = (o1 > p.slots ? p.slots : o1) - b;
                if (n < 0) n = 0;
            }
            begin[e] = (int)b;
            count[e] = (int)n;
            sum += (int)((n + p.MG - 1) / p.MG) * p.n_tiles;
        }
        int run = sum;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int v = __shfl_up_sync(0xFFFFFFFFu, run, d);
            if (lane >= d) run += v;
        }
        int at = run - sum;
        for (int e = lo; e < hi; e++) {
            cum[e] = at;
            at += (count[e] + p.MG - 1) / p.MG * p.n_tiles;
        }
        if (lane == 31) cum[p.E] = run;
        if (bad) raise_status(UW_ERR_DEVICE);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    Plan pl;
    pl.cum = cum;
    pl.begin = begin;
    pl.count = count;
    pl.tiles = cum[p.E];
    {
        const int64_t P = gridDim.x, rounds = pl.tiles / P;
        pl.whole = pl.tiles % P == 0 ? pl.tiles : rounds > 1 ? (rounds - 1) * P : 0;
        pl.units = (pl.tiles - pl.whole) * p.kt;
        // a range shorter than two k steps costs more to join than it saves
        const int64_t most = (pl.units + 1) / 2;
        pl.ps = (int)(P < most ? P : most);
    }
    const int rows_a = p.up ? kTileN / 2 : kTileN;   // outputs of a tile

    if (warp == kProd) {
        // ------------------------------------------------------------ TMA producer
        const bool leader = elect_one();
        Walk wk(pl, blockIdx.x);
        Seg sg;
        Ring r;
        int64_t q = 0;
        bool ok = true;
        while (ok && wk.next(pl, p.kt, sg)) {
            const Tile t = locate(p, pl, sg.tile);
            const int nN = (t.rows + 15) & ~15;
            const int n0 = t.n * rows_a;
            const int64_t wrow = (int64_t)t.e * p.N + n0;
            const int boxes = (nN + p.box - 1) / p.box;
            const uint32_t x_bytes = p.rows ? (uint32_t)nN * 128u * kHalves : (uint32_t)(boxes * p.box) * 128u * kHalves;
            const uint32_t tx = kTileN * kARow + x_bytes + (kMx ? p.sf_a_bytes * (p.up ? 2 : 1) : 0) +
                                (SRC == kGroupMxMx ? p.sf_b_bytes : 0);
            int4 idx[2] = {};
            if (p.rows) {
                // rows past the tile's end repeat its last one (their columns are never stored)
#pragma unroll
                for (int g = 0; g < 2; g++) {
                    int* ip = &idx[g].x;
#pragma unroll
                    for (int i = 0; i < 4; i++) {
                        const int at = 4 * (lane + 32 * g) + i;
                        const int32_t v = p.rows[t.s0 + (at < t.rows ? at : t.rows - 1)];
                        const bool in = v >= 0 && v < p.x_rows;
                        if (!in) raise_status(UW_ERR_DEVICE);
                        ip[i] = in ? v : 0;
                    }
                }
            }
            const uint8_t* sfw = kMx ? p.sw + ((int64_t)t.e * p.w_row_tiles + n0 / kMxTileRows) * p.k_tiles * kMxTileBytes : nullptr;
            const uint8_t* sfu = kMx && p.up ? p.su + ((int64_t)t.e * p.w_row_tiles + n0 / kMxTileRows) * p.k_tiles * kMxTileBytes : nullptr;
            for (int kt = sg.kt0; kt < sg.kt1; kt++, q++, r.advance(p.S)) {
                if (!mbar_wait(empty + 8 * r.i, r.ph ^ 1u, p.timeout, abort_flag)) { ok = false; break; }
                const uint32_t st = base + (uint32_t)r.i * p.stage_bytes, fb = full + 8 * r.i;
                if (leader) {
                    mbar_arrive_expect_tx(fb, tx);
                    const int ax = SRC == kGroupBf16 ? kt * KB : kt * (KB / 2);
                    tma_load_2d(st, &tm_w, ax, (int)wrow, fb);
                    tma_load_2d(st + kTileN / 2 * kARow, p.up ? &tm_u : &tm_w, ax, (int)(p.up ? wrow : wrow + kTileN / 2), fb);
                    if (kMx) {
                        // the stage's part of a scale tile (256 k): all, one half, or the half that holds it
                        const int64_t so = KB == 256 ? (int64_t)kt * kMxTileBytes
                                                     : (int64_t)(KB == 128 ? kt : kt >> 1) * (kMxTileBytes / 2);
                        bulk_load(st + p.off_s, sfw + so, p.sf_a_bytes, fb);
                        if (p.up) bulk_load(st + p.off_s + p.sf_a_bytes, sfu + so, p.sf_a_bytes, fb);
                    }
                    if (SRC == kGroupMxMx) {
                        const int64_t rt = t.s0 / kMxTileRows;
                        for (uint32_t i = 0; i < p.sf_b_bytes / kMxTileBytes; i++) {
                            // a row tile past the last reads the last one again (rows past the end: never stored)
                            const int64_t last = (p.x_rows - 1) / kMxTileRows, at = rt + i < last ? rt + i : last;
                            bulk_load(st + p.off_s + p.sf_a_bytes + i * kMxTileBytes, p.sx + (at * p.k_tiles + kt) * kMxTileBytes,
                                      kMxTileBytes, fb);
                        }
                    }
                    if (!p.rows)
                        for (int h = 0; h < kHalves; h++)
                            for (int b = 0; b < boxes; b++)
                                tma_load_2d(st + p.off_b + (uint32_t)(h * p.MG + b * p.box) * 128u, &tm_x,
                                            SRC == kGroupMxMx ? kt * (KB / 2) : kt * KB + 64 * h, (int)(t.s0 + b * p.box), fb);
                }
                __syncwarp();
                if (p.rows)
#pragma unroll
                    for (int g = 0; g < 2; g++) {
                        const int at = 4 * (lane + 32 * g);
                        if (at < nN)
                            for (int h = 0; h < kHalves; h++)
                                tma_gather4(st + p.off_b + (uint32_t)(h * p.MG + at) * 128u, &tm_x, kt * KB + 64 * h, idx[g], fb);
                    }
            }
        }
        if (!ok)   // every load already issued lands before the CTA exits
            for (int64_t qq = q - p.S < 0 ? 0 : q - p.S; qq < q; qq++)
                mbar_wait(full + 8 * (uint32_t)(qq % p.S), (uint32_t)((qq / p.S) & 1), p.timeout, nullptr);
    } else if (warp == kMma) {
        // ------------------------------------------------------------ MMA issue
        const bool leader = elect_one();
        Walk wk(pl, blockIdx.x);
        Seg sg;
        Ring r, rt, ra;
        bool ok = true;
        while (ok && wk.next(pl, p.kt, sg)) {
            const Tile t = locate(p, pl, sg.tile);
            const int nN = (t.rows + 15) & ~15;
            const uint32_t idesc = mma_idesc_bf16(kTileN, nN);
            if (!mbar_wait(acce + 8 * ra.i, ra.ph ^ 1u, p.timeout, abort_flag)) { ok = false; break; }
            tc_fence_after();
            const uint32_t acc = tmem + (uint32_t)(ra.i * p.MG);
            for (int kt = sg.kt0; kt < sg.kt1; kt++, r.advance(p.S)) {
                if (kRe && !mbar_wait(recon + 8 * rt.i, rt.ph, p.timeout, abort_flag)) { ok = false; break; }
                if (!mbar_wait(full + 8 * r.i, r.ph, p.timeout, abort_flag)) { ok = false; break; }
                tc_fence_after();
                if (leader) {
                    const uint32_t st = base + (uint32_t)r.i * p.stage_bytes;
                    if (SRC == kGroupMxMx) {
                        // scales of the stage: weights 2 x 4 columns, then X 2 x (4 per 128 slots)
                        const uint32_t nb = p.sf_b_bytes / kMxTileBytes;
                        const uint32_t sfa = tmem + p.sf_col0 + (uint32_t)r.i * (8u + 8u * nb), sfb = sfa + 8u;
                        const uint32_t ss = st + p.off_s;
#pragma unroll
                        for (uint32_t h = 0; h < 2; h++) {
                            tc_copy_scales(sfa + 4u * h, ss + 512u * h);
                            for (uint32_t i = 0; i < nb; i++)
                                tc_copy_scales(sfb + 4u * (h * nb + i), ss + p.sf_a_bytes + kMxTileBytes * i + 512u * h);
                        }
                        const uint64_t ad = sw128_desc(st), bd = sw128_desc(st + p.off_b);
#pragma unroll
                        for (uint32_t j = 0; j < 4; j++)
                            tc_mma_mx(acc, ad + 2u * j, bd + 2u * j, idesc_mx(nN, 2u * (j & 1u)), sfa + 4u * (j >> 1),
                                      sfb + 4u * nb * (j >> 1), kt > sg.kt0 || j > 0 ? 1u : 0u);
                    } else {
                        const uint64_t ad = sw128_desc(st);
                        const uint32_t ta = tmem + p.a_col0 + (uint32_t)(KB / 2) * (uint32_t)rt.i;
#pragma unroll
                        for (int h = 0; h < kHalves; h++) {
                            const uint64_t bd = sw128_desc(st + p.off_b + (uint32_t)(h * p.MG) * 128u);
#pragma unroll
                            for (int j = 0; j < 4; j++) {
                                const uint32_t more = kt > sg.kt0 || h > 0 || j > 0 ? 1u : 0u;
                                if (kRe)
                                    tc_mma_tmem_a(acc, ta + 8u * (uint32_t)(4 * h + j), bd + 2u * j, idesc, more);
                                else
                                    tc_mma(acc, ad + 2u * j, bd + 2u * j, idesc, more);
                            }
                        }
                    }
                    tc_commit(empty + 8 * r.i);
                    if (kRe) tc_commit(tfree + 8 * rt.i);
                }
                if (kRe) rt.advance(p.T);
            }
            if (!ok) break;
            if (leader) tc_commit(accf + 8 * ra.i);
            ra.advance(p.nacc);
        }
        // drain the tensor core before tensor memory is released
        if (leader) tc_commit(fin);
        mbar_wait(fin, 0, p.timeout, nullptr);
        __syncwarp();
    } else if (kRe && warp >= kRebuild0) {
        // ------------------------------------------------------------ rebuild
        // Warp w owns tensor-memory lanes (weight rows) 32 (w % 4) ..; the four
        // warps of a quarter (two with two groups) share the stage's pieces of
        // 32 k.  S and T are even with two groups, so a group meets the same
        // slots in every round and sees all their phases in turn.
        constexpr int kPieces = KB / 32;
        constexpr int kPer = kPieces * 4 * kGroups / kRebuildWarps;   // pieces of a warp
        const int rw = warp - kRebuild0, grp = kGroups == 2 ? rw / 8 : 0;
        const int quarter = warp & 3, sub = (kGroups == 2 ? rw % 8 : rw) >> 2;
        const int row = 32 * quarter + lane;
        Walk wk(pl, blockIdx.x);
        Seg sg;
        Ring r, rt;
        bool ok = true;
        while (ok && wk.next(pl, p.kt, sg)) {
            const Tile t = locate(p, pl, sg.tile);
            // where this row's scale bytes are in the stage
            uint32_t so = p.off_s;
            int sq = quarter;
            if (p.up) {
                so += quarter >= 2 ? p.sf_a_bytes : 0;
                sq = (quarter & 1) + (t.n & 1) * 2;
            }
            so += (uint32_t)(lane * 16 + sq * 4);
            for (int kt = sg.kt0; kt < sg.kt1; kt++, r.advance(p.S), rt.advance(p.T)) {
                if (kGroups == 2 && (rt.i & 1) != grp) continue;
                if (!mbar_wait(full + 8 * r.i, r.ph, p.timeout, abort_flag)) { ok = false; break; }
                if (!mbar_wait(tfree + 8 * rt.i, rt.ph ^ 1u, p.timeout, abort_flag)) { ok = false; break; }
                tc_fence_after();
                const uint32_t st = base + (uint32_t)r.i * p.stage_bytes;
#pragma unroll
                for (int i = 0; i < kPer; i++) {
                    const int pc = sub * kPer + i;
                    const uint4 c = lds128(st + swizzled(kARow, row, pc));
                    const int b = KB == 64 ? 2 * (kt & 1) + pc : pc & 3;
                    const uint32_t word = lds32(st + so + (uint32_t)(pc >> 2) * 512u);
                    uint32_t out[16];
                    rebuild32(c, (word >> (8 * b)) & 255u, out);
                    tmem_st16(tmem + p.a_col0 + (uint32_t)(KB / 2) * (uint32_t)rt.i + 16u * (uint32_t)pc +
                                  ((uint32_t)(32 * quarter) << 16),
                              out);
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(recon + 8 * rt.i);
            }
        }
    } else if (warp < 4) {
        // ------------------------------------------------------------ epilogue
        const int row = warp * 32 + lane;
        const uint32_t trow = tmem + ((uint32_t)(warp * 32) << 16);
        const uint32_t stg = base + p.stg_off;
        const size_t slot_f4 = (size_t)(p.MG / 4) * kTileN;   // float4s of a CTA's partial
        Walk wk(pl, blockIdx.x);
        Seg sg;
        Ring ra;
        while (wk.next(pl, p.kt, sg)) {
            const Tile t = locate(p, pl, sg.tile);
            const int nN = (t.rows + 15) & ~15;
            const bool publish = sg.kt0 > 0, joins = sg.kt0 == 0 && sg.kt1 < p.kt;
            int last = blockIdx.x;
            if (joins) last = unit_owner((sg.tile - pl.whole + 1) * p.kt - 1, pl);
            bool good = true;
            for (int b = blockIdx.x + 1; good && b <= last; b++)
                good = wait_tag(p.flags + (size_t)b * 4 + warp, p.epoch, p.timeout, abort_flag);
            if (good) good = mbar_wait(accf + 8 * ra.i, ra.ph, p.timeout, abort_flag, 20000);
            if (any_of_epilogue(!good)) break;
            tc_fence_after();
            const uint32_t acc = trow + (uint32_t)(ra.i * p.MG);
            if (publish) {
                float4* dst = reinterpret_cast<float4*>(p.partial) + (size_t)blockIdx.x * slot_f4 + row;
                for (int c = 0; c < nN; c += 16) {
                    uint32_t v[16];
                    tmem_ld16(acc + (uint32_t)c, v);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 4; i++)
                        __stcg(dst + (size_t)(c / 4 + i) * kTileN,
                               make_float4(__uint_as_float(v[4 * i]), __uint_as_float(v[4 * i + 1]),
                                           __uint_as_float(v[4 * i + 2]), __uint_as_float(v[4 * i + 3])));
                }
                __threadfence();
                __syncwarp();
                if (lane == 0)
                    asm volatile("st.release.gpu.global.u64 [%0], %1;" ::"l"(p.flags + (size_t)blockIdx.x * 4 + warp),
                                 "l"(p.epoch)
                                 : "memory");
            } else {
                const int64_t n0 = (int64_t)t.n * rows_a;
                for (int c0 = 0; c0 < nN; c0 += kChunk) {
                    // accumulator (and the other ranges' partial sums, in k order) -> staging
#pragma unroll
                    for (int hh = 0; hh < 2; hh++) {
                        const int c = c0 + 16 * hh;
                        if (c >= nN) break;
                        uint32_t v[16];
                        tmem_ld16(acc + (uint32_t)c, v);
                        tmem_wait_ld();
                        for (int b = blockIdx.x + 1; b <= last; b++) {
                            const float4* src = reinterpret_cast<const float4*>(p.partial) + (size_t)b * slot_f4 + row;
#pragma unroll
                            for (int i = 0; i < 4; i++) {
                                const float4 x = __ldcg(src + (size_t)(c / 4 + i) * kTileN);
                                v[4 * i] = __float_as_uint(__uint_as_float(v[4 * i]) + x.x);
                                v[4 * i + 1] = __float_as_uint(__uint_as_float(v[4 * i + 1]) + x.y);
                                v[4 * i + 2] = __float_as_uint(__uint_as_float(v[4 * i + 2]) + x.z);
                                v[4 * i + 3] = __float_as_uint(__uint_as_float(v[4 * i + 3]) + x.w);
                            }
                        }
#pragma unroll
                        for (int i = 0; i < 16; i++) sts32(stg + (uint32_t)((16 * hh + i) * kTileN + row) * 4u, v[i]);
                    }
                    named_bar_sync(kEpiBarId, 128);
                    // staging -> Y, 8 outputs a thread
                    const int per = rows_a / 8, cnt = t.rows - c0 < kChunk ? t.rows - c0 : kChunk;
                    for (int i = threadIdx.x; i < cnt * per; i += 128) {
                        const int s = i / per, o = (i % per) * 8;
                        float v[8];
#pragma unroll
                        for (int h = 0; h < 2; h++) {
                            const uint4 x = lds128(stg + (uint32_t)(s * kTileN + o + 4 * h) * 4u);
                            v[4 * h] = __uint_as_float(x.x);
                            v[4 * h + 1] = __uint_as_float(x.y);
                            v[4 * h + 2] = __uint_as_float(x.z);
                            v[4 * h + 3] = __uint_as_float(x.w);
                        }
                        if (p.up) {
#pragma unroll
                            for (int h = 0; h < 2; h++) {
                                const uint4 x = lds128(stg + (uint32_t)(s * kTileN + 64 + o + 4 * h) * 4u);
                                const float u[4] = {__uint_as_float(x.x), __uint_as_float(x.y), __uint_as_float(x.z),
                                                    __uint_as_float(x.w)};
#pragma unroll
                                for (int j = 0; j < 4; j++) {
                                    const float g = v[4 * h + j];
                                    v[4 * h + j] = g / (1.0f + __expf(-g)) * u[j];
                                }
                            }
                        }
                        const int64_t n = n0 + o;
                        const int64_t at = (t.s0 + c0 + s) * p.N + n;
                        if (p.out_f32) {
                            float* y = reinterpret_cast<float*>(p.Y) + at;
                            if (p.y_vec && n + 8 <= p.N) {
                                reinterpret_cast<float4*>(y)[0] = make_float4(v[0], v[1], v[2], v[3]);
                                reinterpret_cast<float4*>(y)[1] = make_float4(v[4], v[5], v[6], v[7]);
                            } else {
#pragma unroll
                                for (int j = 0; j < 8; j++)
                                    if (n + j < p.N) y[j] = v[j];
                            }
                        } else {
                            uint16_t* y = reinterpret_cast<uint16_t*>(p.Y) + at;
                            if (p.y_vec && n + 8 <= p.N) {
                                *reinterpret_cast<uint4*>(y) =
                                    make_uint4(bf2(v[0], v[1]), bf2(v[2], v[3]), bf2(v[4], v[5]), bf2(v[6], v[7]));
                            } else {
#pragma unroll
                                for (int j = 0; j < 8; j++)
                                    if (n + j < p.N) y[j] = bf(v[j]);
                            }
                        }
                    }
                    named_bar_sync(kEpiBarId, 128);
                }
                // the tags are cleared for a replay of this call
                if (lane == 0)
                    for (int b = blockIdx.x + 1; b <= last; b++) p.flags[(size_t)b * 4 + warp] = 0ull;
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(acce + 8 * ra.i);
            ra.advance(p.nacc);
        }
    }

    tc_fence_before();
    __syncthreads();
    if (*abort_flag && threadIdx.x == 0) raise_status(UW_ERR_TIMEOUT);
    if (warp == kMma) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

__global__ void __launch_bounds__(kThreadsPlain, 1)
    k_group_bf16(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w,
                 const __grid_constant__ CUtensorMap tm_u, const GroupParams p) {
    group_body<kGroupBf16, 64>(tm_x, tm_w, tm_u, p);
}

__global__ void __launch_bounds__(kThreadsPlain, 1)
    k_group_mx_mx(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w,
                  const __grid_constant__ CUtensorMap tm_u, const GroupParams p) {
    group_body<kGroupMxMx, 256>(tm_x, tm_w, tm_u, p);
}

// 22 warps: 16 K registers of a sub-partition over six of them allow 80.
template <int KB>
__global__ void __maxnreg__(80)
    k_group_mx(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w,
               const __grid_constant__ CUtensorMap tm_u, const GroupParams p) {
    group_body<kGroupMx, KB>(tm_x, tm_w, tm_u, p);
}

// Slots of a tile: twice the mean group (groups are uneven), a power of two
// from 16 to 256.  Block-scaled products keep 128-slot scale tiles whole.
int pick_tile_slots(int src, int64_t slots, int E) {
    const int64_t groups = E < slots ? E : slots;
    const int64_t mean = (slots + groups - 1) / groups;
    const int64_t want = E == 1 ? mean : 2 * mean;
    int mg = src == kGroupMxMx ? 128 : 16;
    while (mg < 256 && mg < want) mg *= 2;
    return mg;
}

}  // namespace

size_t group_ws_bytes(int src, int64_t slots, int E) {
    if (slots <= 0) return 0;
    const int P = num_sms(), mg = pick_tile_slots(src, slots, E);
    return (size_t)P * mg * kTileN * 4 + (((size_t)P * 4 * 8 + 255) & ~size_t(255));
}

cudaError_t launch_group(const GroupGemm& a, cudaStream_t s, uw_status* st) {
    *st = UW_OK;
    if (a.slots == 0) return cudaSuccess;
    GroupParams p{};
    const int MG = pick_tile_slots(a.src, a.slots, a.E);
    const int KB = a.src == kGroupBf16 ? 64 : a.src == kGroupMxMx ? 256 : MG <= 32 ? 256 : MG <= 128 ? 128 : 64;
    p.x_rows = a.x_rows;
    p.slots = a.slots;
    p.N = a.N;
    p.rows = a.rows;
    p.offsets = a.offsets;
    p.E = a.E;
    p.kt = (int)((a.K + KB - 1) / KB);
    p.MG = MG;
    p.box = MG < 64 ? MG : 64;
    p.up = a.up ? 1 : 0;
    const int rows_a = p.up ? kTileN / 2 : kTileN;
    p.n_tiles = (int)((a.N + rows_a - 1) / rows_a);
    const int64_t max_tiles = ((a.slots + MG - 1) / MG + a.E) * (int64_t)p.n_tiles;
    if (max_tiles > 0x7FFFFFFF) { *st = UW_ERR_SHAPE; return cudaSuccess; }
    p.out_f32 = a.out_f32;
    p.y_vec = a.N % 8 == 0;
    p.Y = a.Y;
    p.sw = a.w_scales;
    p.su = a.up_scales;
    p.sx = a.x_scales;
    p.w_row_tiles = mx_row_tiles(a.N);
    p.k_tiles = (int)mx_k_tiles(a.K);
    const int P = num_sms();
    if (!a.ws || a.ws_bytes < group_ws_bytes(a.src, a.slots, a.E)) { *st = UW_ERR_WORKSPACE; return cudaSuccess; }
    p.partial = (float*)a.ws;
    p.flags = (unsigned long long*)((uint8_t*)a.ws + (size_t)P * MG * kTileN * 4);
    p.epoch = gemm_next_epoch();
    p.timeout = timeout_ns();

    // stage: weight rows, scale bytes, X (every swizzled tile 1024-byte aligned)
    auto al1k = [](uint32_t x) { return (x + 1023u) & ~1023u; };
    const uint32_t a_row = a.src == kGroupBf16 ? 128 : KB / 2;
    const int halves = a.src == kGroupMxMx ? 1 : KB / 64;
    p.off_s = kTileN * a_row;
    p.sf_a_bytes = a.src == kGroupBf16 ? 0 : KB == 256 ? kMxTileBytes : kMxTileBytes / 2;
    p.sf_b_bytes = a.src == kGroupMxMx ? (uint32_t)(MG / kMxTileRows) * kMxTileBytes : 0;
    p.off_b = al1k(p.off_s + p.sf_a_bytes * (p.up ? 2 : 1) + p.sf_b_bytes);
    p.stage_bytes = p.off_b + (uint32_t)(MG * 128 * halves);
    const uint32_t ctrl = 512, tab = (uint32_t)(3 * a.E + 1) * 4;
    const uint32_t fixed = 1024 + ctrl + kStage32 + ((tab + 15u) & ~15u);
    // tensor memory: accumulators, then rebuilt-A slots (KB/2 columns) or scale columns
    const uint32_t per_slot = a.src == kGroupMx ? KB / 2 : a.src == kGroupMxMx ? 8 + 8 * (MG / kMxTileRows) : 0;
    p.nacc = a.src == kGroupBf16 || 2 * MG <= 256 ? 2 : 1;
    const uint32_t acc_cols = (uint32_t)(p.nacc * MG);
    int S = (int)((227 * 1024 - fixed) / p.stage_bytes);
    if (S > kMaxS) S = kMaxS;
    if (a.src == kGroupMxMx && S > (int)((kTmemCols - acc_cols) / per_slot)) S = (int)((kTmemCols - acc_cols) / per_slot);
    p.T = 0;
    if (a.src == kGroupMx) {
        p.T = (int)((kTmemCols - acc_cols) / per_slot);
        if (p.T > kMaxT) p.T = kMaxT;
        if (KB == 64) {   // two rebuild groups: even rings
            S &= ~1;
            p.T &= ~1;
        }
    }
    if (S < 2 || (a.src == kGroupMx && p.T < 2)) { *st = UW_ERR_UNSUPPORTED; return cudaSuccess; }
    p.S = S;
    p.a_col0 = p.sf_col0 = acc_cols;
    p.ctrl_off = (uint32_t)S * p.stage_bytes;
    p.stg_off = p.ctrl_off + ctrl;
    p.tab_off = p.stg_off + kStage32;
    const size_t smem = (size_t)S * p.stage_bytes + fixed;

    CUtensorMap tx{}, tw{}, tu{};
    bool ok;
    const uint64_t wrows = (uint64_t)a.E * (uint64_t)a.N;
    if (a.src == kGroupMxMx)
        ok = make_map_2d(&tx, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, a.X, a.K / 2, a.x_rows, a.K / 2, 128, p.box,
                         CU_TENSOR_MAP_SWIZZLE_128B);
    else
        ok = make_map_2d(&tx, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, a.X, a.K, a.x_rows, a.K * 2, 64, a.rows ? 1 : p.box,
                         CU_TENSOR_MAP_SWIZZLE_128B);
    for (int h = 0; h < 2; h++) {
        const void* w = h && a.up ? a.up : a.W;
        CUtensorMap* m = h ? &tu : &tw;
        if (a.src == kGroupBf16)
            ok = ok && make_map_2d(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, w, a.K, wrows, a.K * 2, 64, kTileN / 2,
                                   CU_TENSOR_MAP_SWIZZLE_128B);
        else
            ok = ok && make_map_2d(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, w, a.K / 2, wrows, a.K / 2, a_row, kTileN / 2,
                                   KB == 256   ? CU_TENSOR_MAP_SWIZZLE_128B
                                   : KB == 128 ? CU_TENSOR_MAP_SWIZZLE_64B
                                               : CU_TENSOR_MAP_SWIZZLE_32B);
    }
    if (!ok) { *st = UW_ERR_CUDA; return cudaSuccess; }

    void (*kern)(const CUtensorMap, const CUtensorMap, const CUtensorMap, const GroupParams) =
        a.src == kGroupBf16   ? k_group_bf16
        : a.src == kGroupMxMx ? k_group_mx_mx
        : KB == 256           ? k_group_mx<256>
        : KB == 128           ? k_group_mx<128>
                              : k_group_mx<64>;
    cudaError_t e = set_smem_attr((const void*)kern, (int)smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(max_tiles * p.kt < P ? max_tiles * p.kt : P));
    cfg.blockDim = dim3(a.src == kGroupMx ? kThreadsRebuild : kThreadsPlain);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, kern, tx, tw, tu, p);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace uw
