// uw_route.cu -- the ends of an expert layer: the router's choice with the
// slots sorted by expert, and the weighted sum of the experts' outputs.
//
// Router.  The choice compares logits only (softmax and sigmoid rise with
// the logit), by an order-preserving 32-bit key, so it is exact whatever the
// scores round to.  A token has G lanes, E/G keys each: 8 lanes (four tokens a
// warp) up to 256 experts and 8 choices, else a warp.  k rounds take the
// largest key; a round costs a lane one instruction a key, so few lanes with
// many keys share its reductions best (16384 tokens, 256 experts, k = 8, BF16:
// 22.9 us with a warp a token, 17.7 us with 8 lanes).  Scores are fp32 with the accurate
// exponential.
// Slots.  A stable counting sort over at most one CTA per SM: CTA b owns a
// contiguous run of tokens, counts its choices per expert (k_route_choose),
// and after all counts are known (k_route_place) adds up the counts of the
// CTAs before it, the experts before each expert and, inside the CTA, of the
// warps before each warp.  Ranks inside a warp come from match_any, so the
// order -- and every output -- is the same on every run.  What bounds it: the
// logits are read once; below a few thousand tokens the launches' latency.
// With few choices one CTA does both parts in a single launch.  Measured: 16
// tokens of 64 experts, k = 6: 5.3 us; 16384 tokens of 256 experts in fp32, k = 8:
// 24 us against 2.9 us for the bytes: latency (profiled apart the choice takes 20
// us, 9 chained rounds of 32 keys a lane at 40 % issue and 11 % of DRAM, and the
// places 17 us at 32 % issue; the second's start overlaps).
//
// Combination.  Y[t] = sum_j w[t,j] Z[pos[t,j]]: bound by reading T k N and
// writing T N values once.  A warp owns 256 columns of one token at a time, 8 a
// lane; lane j holds choice j, and the next item's choices are loaded before
// the eight rows in flight are added.  Measured: 8192 tokens of 8 rows of 4096 in
// BF16: 100 us, 6.1 TB/s; 8 tokens of 2 rows: 2.5 us.
#include "uw_device.cuh"
#include "uw_internal.h"

namespace uw {

int route_status_take() { return unit_status_take(); }

namespace {

constexpr int kRouteThreads = 1024;   // at most
constexpr uint32_t kFull = 0xFFFFFFFFu;
constexpr int kSingle = 512;     // choices up to which one CTA does everything

struct RouteParams {
    const void* logits;
    int64_t T;
    int E, k, score, renorm;
    int vec;         // rows of four logits a load (E % 4 = 0, aligned)
    float scale;
    int64_t chunk;   // tokens of a CTA
    int32_t* ids;
    float* weights;
    int32_t* offsets;
    int32_t* rows;
    int32_t* pos;
    int32_t* hist;   // [CTAs][E]
};

__device__ __forceinline__ float key_logit(uint32_t k) {
    return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}

// Over the G lanes of a token.
template <int G>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int d = G / 2; d; d >>= 1) v += __shfl_xor_sync(kFull, v, d);
    return v;
}
template <int G>
__device__ __forceinline__ uint32_t group_max(uint32_t v) {
    if constexpr (G == 32) {
        return __reduce_max_sync(kFull, v);
    } else {
#pragma unroll
        for (int d = G / 2; d; d >>= 1) {
            const uint32_t o = __shfl_xor_sync(kFull, v, d);
            v = v > o ? v : o;
        }
        return v;
    }
}

// Expert of a lane's key i: four neighbours a load where the lane has so many.
template <int VPL, int G>
__device__ __forceinline__ constexpr int expert_of(int i, int lane) {
    return VPL % 4 ? G * i + lane : 4 * G * (i / 4) + 4 * lane + i % 4;
}

// Logits of token t as fp32 bits (NaN past E and for the lanes without a
// token); all loads are issued before any is used.
template <int VPL, int G, bool F32>
__device__ __forceinline__ void load_logits(const RouteParams& p, int64_t t, bool in, int lane, uint32_t (&raw)[VPL]) {
    const uint32_t* x = reinterpret_cast<const uint32_t*>(p.logits) + t * p.E;
    const uint16_t* h = reinterpret_cast<const uint16_t*>(p.logits) + t * p.E;
    if constexpr (VPL % 4 == 0) {
        if (p.vec) {
#pragma unroll
            for (int i = 0; i < VPL; i += 4) {
                const int e = expert_of<VPL, G>(i, lane);
                const bool ok = in && e < p.E;
                if (F32) {
                    const uint4 v = ok ? __ldg(reinterpret_cast<const uint4*>(x + e)) : make_uint4(0x7FC00000u, 0x7FC00000u, 0x7FC00000u, 0x7FC00000u);
                    raw[i] = v.x;
                    raw[i + 1] = v.y;
                    raw[i + 2] = v.z;
                    raw[i + 3] = v.w;
                } else {
                    const uint2 v = ok ? __ldg(reinterpret_cast<const uint2*>(h + e)) : make_uint2(0x7FC07FC0u, 0x7FC07FC0u);
                    raw[i] = v.x << 16;
                    raw[i + 1] = v.x & 0xFFFF0000u;
                    raw[i + 2] = v.y << 16;
                    raw[i + 3] = v.y & 0xFFFF0000u;
                }
            }
            return;
        }
    }
#pragma unroll
    for (int i = 0; i < VPL; i++) {
        const int e = expert_of<VPL, G>(i, lane);
        const bool ok = in && e < p.E;
        if (F32) raw[i] = ok ? __ldg(x + e) : 0x7FC00000u;
        else raw[i] = ok ? (uint32_t)__ldg(h + e) << 16 : 0x7FC00000u;
    }
}

// Order-preserving key of a logit's bits; 0: never chosen (NaN, -infinity).
// +infinity counts as the largest finite number, -0 as 0.
__device__ __forceinline__ uint32_t bits_key(uint32_t bits) {
    const uint32_t b = __float_as_uint(__uint_as_float(bits) + 0.0f);   // -0 -> 0, every NaN -> a positive one
    const uint32_t k = b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
    const uint32_t top = 0xFF7FFFFFu;                                    // the largest finite number's
    // -infinity: 0x007FFFFF; numbers from 0x00800000; infinity: 0xFF800000; NaN above
    return k - 0x00800000u > 0xFF800000u - 0x00800000u ? 0u : k < top ? k : top;
}

// Where the last choice shares its upper key bits (`prefix`) with keys that
// were left out: the choices first .. k - 1 of the token are the largest of all
// keys with that prefix, equal keys by index.  Lane j of the G lanes with first
// <= j < k ends up with choice j as (expert, key).  `on`: the token needs it
// (every lane of the warp takes part).
template <int VPL, int G, int BITS>
__device__ __noinline__ uint2 select_edge(const RouteParams& p, int64_t t, bool on, int lane, uint32_t prefix, int first) {
    uint32_t key[VPL];
    load_logits<VPL, G, true>(p, t, on, lane, key);
#pragma unroll
    for (int i = 0; i < VPL; i++) {
        key[i] = bits_key(key[i]);
        if ((key[i] >> BITS) != prefix) key[i] = 0;
    }
    uint2 mine = make_uint2(0xFFFFFFFFu, 0);
    for (int j = on ? first : p.k; __any_sync(kFull, j < p.k); j++) {
        uint32_t best = 0, cand = 0;
#pragma unroll
        for (int i = 0; i < VPL; i++) best = best > key[i] ? best : key[i];
        const uint32_t mx = group_max<G>(best);
#pragma unroll
        for (int i = VPL - 1; i >= 0; i--)
            if (key[i] == mx) cand = (uint32_t)(0x7FFFFFFF - expert_of<VPL, G>(i, lane));   // the lowest index has the largest
        const uint32_t e = 0x7FFFFFFFu - group_max<G>(cand);
#pragma unroll
        for (int i = 0; i < VPL; i++)
            if ((uint32_t)expert_of<VPL, G>(i, lane) == e) key[i] = 0;
        if (lane == j && mx) mine = make_uint2(e, mx);
    }
    return mine;
}

// One token: lane j < k ends up with choice j (expert id, or -1) and weight.
// The rounds run on words that join a key's upper bits with the index in the
// lower ones (as many as VPL G experts need): one maximum a round, and the word
// that gave it is unique.  The upper bits hold all of a BF16 logit.  fp32
// logits may differ below them: where two neighbours among the choices share
// them (about 1 token in 200 at 256 experts) the choices are put in order by
// their full keys; where the last choice shares them with the first one left
// out (1 in 1500), the keys that share them are selected exactly first.
template <int VPL, int G, bool F32>
__device__ __forceinline__ void choose(const RouteParams& p, int64_t t, bool in, uint32_t (&word)[VPL], int lane, int& id,
                                       float& w) {
    constexpr int kBits = VPL * G <= 32 ? 5 : VPL * G <= 64 ? 6 : VPL * G <= 128 ? 7 : VPL * G <= 256 ? 8 : VPL * G <= 512 ? 9 : 10;
    constexpr uint32_t kLow = (1u << kBits) - 1u;
    uint32_t best = 0;
    float total = 0.0f, m = 0.0f;
#pragma unroll
    for (int i = 0; i < VPL; i++) word[i] = bits_key(word[i]);
    if (p.score == UW_SCORE_SOFTMAX) {
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < VPL; i++) top = top > word[i] ? top : word[i];
        top = group_max<G>(top);
        m = key_logit(top);   // top = 0 (no choice at all): unused
        if (!p.renorm) {   // the denominator over every logit
#pragma unroll
            for (int i = 0; i < VPL; i++)
                if (word[i]) total += expf(key_logit(word[i]) - m);
            total = group_sum<G>(total);
        }
    }
#pragma unroll
    for (int i = 0; i < VPL; i++) {
        word[i] = word[i] ? (word[i] & ~kLow) | (kLow - (uint32_t)expert_of<VPL, G>(i, lane)) : 0u;
        best = best > word[i] ? best : word[i];
    }
    uint32_t got = 0, last = 0;
    bool close = false, edge = false;
    for (int j = 0;; j++) {
        const uint32_t mx = group_max<G>(best);
        // fp32: a word that shares its key bits with the one before (also the first that is not taken)
        if (F32) edge = j && mx && (mx >> kBits) == (last >> kBits);
        if (j == p.k) break;
        close |= edge;
        last = mx;
        if (lane == j) got = mx;
        if (!F32 && j + 1 == p.k) break;
        // the largest word below mx: word - mx wraps to the top of the range below it, to its bottom from it up
        uint32_t below = 0;
#pragma unroll
        for (int i = 0; i < VPL; i++) below = __viaddmax_u32(word[i], 0u - mx, below);
        best = below + mx;
        best = mx && best < mx ? best : 0u;
    }
    id = got ? (int)(kLow - (got & kLow)) : -1;
    uint32_t mine = 0;
    if (!F32) {
        mine = got & ~kLow;
        // A BF16 logit's key ends in 16 zeros, a negative one's in 16 ones, and so does that of +infinity, which counts as
        // the largest fp32 number: the softmax subtracts that very number.
        if (mine & 0xFFFFu) mine |= kLow;
    } else {
        if (id >= 0) mine = bits_key(__ldg(reinterpret_cast<const uint32_t*>(p.logits) + t * p.E + id));
        if (__any_sync(kFull, edge)) {
            // choices above the prefix that the last one shares stand
            const uint32_t prefix = last >> kBits;
            const uint32_t above = __ballot_sync(kFull, got && (got >> kBits) > prefix);
            const int first = __popc(G == 32 ? above : above >> ((threadIdx.x & 31) / G * G) & ((1u << (G % 32)) - 1u));
            const uint2 x = select_edge<VPL, G, kBits>(p, t, edge, lane, prefix, first);
            if (edge && lane >= first && lane < p.k) {
                id = (int)x.x;
                mine = x.y;
            }
        }
        if (__any_sync(kFull, close || edge)) {   // by (key, index): every lane's place among the choices, then the choice of each place
            int place = 0, from = lane;
            for (int i = 0; i < p.k; i++) {
                const uint32_t k = __shfl_sync(kFull, mine, i, G);
                const int e = __shfl_sync(kFull, id, i, G);
                place += k > mine || (k == mine && (uint32_t)e < (uint32_t)id);
            }
            for (int i = 0; i < p.k; i++)
                if (__shfl_sync(kFull, place, i, G) == lane) from = i;
            // (empty choices, key 0, share a place behind all others: they stay where they are)
            const uint32_t k = __shfl_sync(kFull, mine, from, G);
            const int e = __shfl_sync(kFull, id, from, G);
            if (mine) {
                mine = k;
                id = e;
            }
        }
    }
    const float x = key_logit(mine);
    float s = 0.0f;
    if (mine) s = p.score == UW_SCORE_SOFTMAX ? expf(x - m) : 1.0f / (1.0f + expf(-x));
    if (p.renorm) total = group_sum<G>(s);
    if (p.score == UW_SCORE_SOFTMAX || p.renorm) s = total > 0.0f ? s / total : 0.0f;
    w = mine ? s * p.scale : 0.0f;
}

// Positions of the CTA's choices, the offsets (CTA 0) and the rows of the
// slots.  `sm` holds base[E], total[E + 1] and wcount[warps][E].  A single CTA
// brings its own counts and choices in shared memory, else they are read from
// what k_route_choose wrote.
__device__ __forceinline__ void place(const RouteParams& p, int32_t* sm, int ctas, const int32_t* counts, const int32_t* ids) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, E = p.E, threads = blockDim.x, warps = threads >> 5;
    int32_t* base = sm;
    int32_t* total = sm + E;
    int32_t* wcount = total + E + 1;
    for (int i = tid; i < 2 * E + 1 + warps * E; i += threads) sm[i] = 0;
    // a warp owns a contiguous run of the CTA's entries; its first 32 are read once
    const int64_t t0 = (int64_t)blockIdx.x * p.chunk;
    const int64_t t1 = t0 + p.chunk < p.T ? t0 + p.chunk : p.T;
    const int64_t first = t0 * p.k;
    const int64_t n = t1 > t0 ? (t1 - t0) * p.k : 0;
    const int64_t per = ((n + warps - 1) / warps + 31) / 32 * 32;
    const int64_t lo = per * warp, hi = per * (warp + 1);
    const int64_t w0 = first + (lo < n ? lo : n), w1 = first + (hi < n ? hi : n);
    if (!counts) {
        asm volatile("griddepcontrol.wait;" ::: "memory");
        asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    }
    const int e0 = w0 + lane < w1 ? ids[w0 + lane] : -1;
    __syncthreads();
    if (counts) {
        for (int e = tid; e < E; e += threads) total[e] = counts[e];
    } else {
        // counts of the CTAs before this one, and of all: the threads cover E
        // experts times as many row groups as fit
        const int groups = threads / E > 1 ? threads / E : 1;
        if (tid < groups * E) {   // E <= threads
            const int e = tid % E, g = tid / E;
            int before = 0, all = 0;
#pragma unroll 16
            for (int b = g; b < ctas; b += groups) {
                const int c = __ldcg(p.hist + (int64_t)b * E + e);
                all += c;
                before += b < (int)blockIdx.x ? c : 0;
            }
            if (before) atomicAdd(&base[e], before);
            if (all) atomicAdd(&total[e], all);
        }
    }
    int32_t* mine = wcount + warp * E;
    if (e0 >= 0) atomicAdd(&mine[e0], 1);
    for (int64_t i = w0 + 32 + lane; i < w1; i += 32) {
        const int e = ids[i];
        if (e >= 0) atomicAdd(&mine[e], 1);
    }
    __syncthreads();
    // exclusive prefix of the totals over the experts (warp 0, E/32 each)
    if (warp == 0) {
        const int each = (E + 31) / 32, lo = lane * each < E ? lane * each : E, hi = lo + each < E ? lo + each : E;
        int sum = 0;
        for (int e = lo; e < hi; e++) sum += total[e];
        int run = sum;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int v = __shfl_up_sync(kFull, run, d);
            if (lane >= d) run += v;
        }
        int at = run - sum;
        for (int e = lo; e < hi; e++) {
            const int c = total[e];
            total[e] = at;
            at += c;
        }
        if (lane == 31) total[E] = run;
    }
    __syncthreads();
    // first slot of every warp and expert: the warps' counts of an expert are
    // scanned by `share` neighbouring lanes, kRankWarps / share rows each
    {
        int share = 1;
        while (2 * share <= warps && 2 * share * E <= threads) share *= 2;
        const int rows = (warps + share - 1) / share;
        for (int i0 = 0; i0 < E * share; i0 += threads) {   // one round but for a small single CTA
            const int i = i0 + tid, e = i / share, part = i % share, r0 = part * rows;
            const int r1 = e >= E ? r0 : r0 + rows < warps ? r0 + rows : warps;
            int sum = 0;
            for (int w = r0; w < r1; w++) sum += wcount[w * E + e];
            int run = sum;
            for (int d = 1; d < share; d <<= 1) {
                const int v = __shfl_up_sync(kFull, run, d, share);
                if (part >= d) run += v;
            }
            int at = e < E ? total[e] + base[e] + run - sum : 0;
            for (int w = r0; w < r1; w++) {
                const int c = wcount[w * E + e];
                wcount[w * E + e] = at;
                at += c;
            }
        }
    }
    if (blockIdx.x == 0)
        for (int e = tid; e <= E; e += threads) p.offsets[e] = total[e];
    __syncthreads();
    for (int64_t i0 = w0; i0 < w1; i0 += 32) {
        const int64_t i = i0 + lane;
        const int e = i0 == w0 ? e0 : i < w1 ? ids[i] : -1;
        const uint32_t same = __match_any_sync(kFull, e);
        int slot = -1;
        if (e >= 0) slot = mine[e] + __popc(same & ((1u << lane) - 1u));
        __syncwarp();
        if (e >= 0 && lane == 31 - __clz(same)) mine[e] = slot + 1;
        __syncwarp();
        if (i < w1) {
            p.pos[i] = slot;
            if (slot >= 0) p.rows[slot] = (int32_t)((uint32_t)i / (uint32_t)p.k);   // T k < 2^31
        }
    }
    // slots that no choice fills
    const int64_t all = p.T * p.k;
    for (int64_t i = total[E] + (int64_t)blockIdx.x * threads + tid; i < all; i += (int64_t)ctas * threads)
        p.rows[i] = -1;
}

template <int VPL, int G, bool F32>
__global__ void __launch_bounds__(kRouteThreads) k_route_choose(const RouteParams p) {
    extern __shared__ int32_t sm[];
    int32_t* counts = sm;
    int32_t* ids = sm + p.E;   // a single CTA keeps its choices here too
    const bool single = gridDim.x == 1;
    const int threads = blockDim.x, warps = threads >> 5;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int e = threadIdx.x; e < p.E; e += threads) counts[e] = 0;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    __syncthreads();
    const int64_t t0 = (int64_t)blockIdx.x * p.chunk;
    const int64_t t1 = t0 + p.chunk < p.T ? t0 + p.chunk : p.T;
    // a warp takes 32 / G tokens at a time
    constexpr int kTok = 32 / G;
    const int gl = lane % G;
    for (int64_t tw = t0 + (int64_t)warp * kTok; tw < t1; tw += (int64_t)warps * kTok) {
        const int64_t t = tw + lane / G;
        const bool in = t < t1;
        uint32_t raw[VPL];
        load_logits<VPL, G, F32>(p, t, in, gl, raw);
        int id;
        float w;
        choose<VPL, G, F32>(p, t, in, raw, gl, id, w);
        if (in && gl < p.k) {
            p.ids[t * p.k + gl] = id;
            p.weights[t * p.k + gl] = w;
            if (id >= 0) atomicAdd(&counts[id], 1);
            if (single) ids[t * p.k + gl] = id;
        }
    }
    __syncthreads();
    if (single)
        place(p, ids + kSingle, 1, counts, ids);
    else
        for (int e = threadIdx.x; e < p.E; e += threads) p.hist[(int64_t)blockIdx.x * p.E + e] = counts[e];
}

__global__ void __launch_bounds__(kRouteThreads) k_route_place(const RouteParams p) {
    extern __shared__ int32_t sm[];
    place(p, sm, (int)gridDim.x, nullptr, p.ids);
}

template <typename P>
cudaError_t launch_pdl(void (*kern)(const P), int64_t grid, int threads, size_t smem, cudaStream_t s, const P& p) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, kern, p);
    return e != cudaSuccess ? e : cudaGetLastError();
}

typedef void (*RouteKernel)(const RouteParams);
// (a warp a token while an SM has fewer than 16 tokens: then the rounds' latency counts)
bool eight_lanes(int64_t T, int E, int k, int ctas) { return E <= 256 && k <= 8 && T >= 16 * (int64_t)ctas && ctas > 1; }
template <bool F32>
RouteKernel route_kernel(int E, bool eight) {
    if (eight)
        return E <= 32    ? k_route_choose<4, 8, F32>
               : E <= 64  ? k_route_choose<8, 8, F32>
               : E <= 128 ? k_route_choose<16, 8, F32>
                          : k_route_choose<32, 8, F32>;
    return E <= 32    ? k_route_choose<1, 32, F32>
           : E <= 64  ? k_route_choose<2, 32, F32>
           : E <= 128 ? k_route_choose<4, 32, F32>
           : E <= 256 ? k_route_choose<8, 32, F32>
           : E <= 512 ? k_route_choose<16, 32, F32>
                      : k_route_choose<32, 32, F32>;
}

// ---------------------------------------------------------------- combination
constexpr int kCombineThreads = 256;
constexpr int kCombineCols = 8;     // columns of a thread
constexpr int kCombineAhead = 8;    // rows in flight

struct CombineParams {
    const void* Z;
    int64_t slots;
    const int32_t* pos;
    const float* weights;
    int64_t T;
    int k;
    int64_t N;
    int64_t groups;   // column groups of 256
    void* Y;
};

// 8 columns as loaded: BF16 in the first vector, fp32 in both.
template <bool F32>
struct Cols {
    uint4 a, b;
};

template <bool F32>
__device__ __forceinline__ void load_cols(const void* Z, int64_t at, int n, bool vec, Cols<F32>& r) {
    if (vec) {
        const uint4* z = F32 ? reinterpret_cast<const uint4*>(reinterpret_cast<const float*>(Z) + at)
                             : reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(Z) + at);
        r.a = __ldcs(z);
        if (F32) r.b = __ldcs(z + 1);
    } else {
        uint32_t w[8] = {};
#pragma unroll
        for (int i = 0; i < 8; i++)
            if (i < n) {
                if (F32) w[i] = reinterpret_cast<const uint32_t*>(Z)[at + i];
                else w[i >> 1] |= (uint32_t) reinterpret_cast<const uint16_t*>(Z)[at + i] << (16 * (i & 1));
            }
        r.a = make_uint4(w[0], w[1], w[2], w[3]);
        if (F32) r.b = make_uint4(w[4], w[5], w[6], w[7]);
    }
}

template <bool F32>
__device__ __forceinline__ void add_cols(const Cols<F32>& r, float w, float (&acc)[8]) {
    const uint32_t a[4] = {r.a.x, r.a.y, r.a.z, r.a.w}, b[4] = {r.b.x, r.b.y, r.b.z, r.b.w};
#pragma unroll
    for (int i = 0; i < 4; i++) {
        if (F32) {
            acc[i] = fmaf(w, __uint_as_float(a[i]), acc[i]);
            acc[4 + i] = fmaf(w, __uint_as_float(b[i]), acc[4 + i]);
        } else {
            acc[2 * i] = fmaf(w, __uint_as_float(a[i] << 16), acc[2 * i]);
            acc[2 * i + 1] = fmaf(w, __uint_as_float(a[i] & 0xFFFF0000u), acc[2 * i + 1]);
        }
    }
}

// Rows of N values are 16-byte aligned runs of 8 columns when N % 8 == 0;
// otherwise every value is loaded and stored by itself.
template <bool IN32, bool OUT32>
__global__ void __launch_bounds__(kCombineThreads, IN32 ? 2 : 4) k_combine(const CombineParams p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int lane = threadIdx.x & 31;
    const int64_t warps = (int64_t)gridDim.x * (kCombineThreads / 32), items = p.T * p.groups;
    int64_t i = (int64_t)blockIdx.x * (kCombineThreads / 32) + (threadIdx.x >> 5);
    const bool vec = p.N % 8 == 0;
    bool wrong = false;
    int32_t s_next = -1;
    float w_next = 0.0f;
    auto choice = [&](int64_t item) {   // lane j: choice j of the item's token
        s_next = -1;
        w_next = 0.0f;
        if (item < items && lane < p.k) {
            const int64_t at = item / p.groups * p.k + lane;
            s_next = __ldg(p.pos + at);
            w_next = __ldg(p.weights + at);
            if (s_next >= p.slots) {
                wrong = true;
                s_next = -1;
            }
        }
    };
    choice(i);
    for (; i < items; i += warps) {
    const int64_t t = i / p.groups, c = (i - t * p.groups) * (32 * kCombineCols) + lane * kCombineCols;
    const int n = p.N - c < 8 ? (int)(p.N - c) : 8;   // columns of this lane (none or less than none: past the row)
    const int32_t s_mine = s_next;
    const float w_mine = w_next;
    float acc[8] = {};
    for (int j0 = 0; j0 < p.k; j0 += kCombineAhead) {
        Cols<IN32> z[kCombineAhead];
#pragma unroll
        for (int j = 0; j < kCombineAhead; j++) {
            const int32_t s = j0 + j < p.k ? __shfl_sync(kFull, s_mine, j0 + j) : -1;
            z[j].a = z[j].b = make_uint4(0, 0, 0, 0);
            if (s >= 0 && n > 0) load_cols<IN32>(p.Z, s * p.N + c, n, vec, z[j]);
        }
        if (j0 == 0) choice(i + warps);   // meanwhile
#pragma unroll
        for (int j = 0; j < kCombineAhead; j++) {
            if (j0 + j >= p.k) break;
            const int32_t s = __shfl_sync(kFull, s_mine, j0 + j);
            const float w = __shfl_sync(kFull, w_mine, j0 + j);
            add_cols<IN32>(z[j], s < 0 ? 0.0f : w, acc);
        }
    }
    if (n <= 0) continue;
    const int64_t at = t * p.N + c;
    if (OUT32) {
        float* y = reinterpret_cast<float*>(p.Y) + at;
        if (vec) {
            __stcs(reinterpret_cast<float4*>(y), make_float4(acc[0], acc[1], acc[2], acc[3]));
            __stcs(reinterpret_cast<float4*>(y) + 1, make_float4(acc[4], acc[5], acc[6], acc[7]));
        } else {
#pragma unroll
            for (int q = 0; q < 8; q++)
                if (q < n) y[q] = acc[q];
        }
    } else {
        __nv_bfloat16* y = reinterpret_cast<__nv_bfloat16*>(p.Y) + at;
        if (vec) {
            uint4 o;
            uint32_t* op = &o.x;
#pragma unroll
            for (int q = 0; q < 4; q++) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(acc[2 * q], acc[2 * q + 1]);
                op[q] = *reinterpret_cast<const uint32_t*>(&h);
            }
            __stcs(reinterpret_cast<uint4*>(y), o);
        } else {
#pragma unroll
            for (int q = 0; q < 8; q++)
                if (q < n) y[q] = __float2bfloat16_rn(acc[q]);
        }
    }
    }
    if (wrong) raise_status(UW_ERR_DEVICE);
}

}  // namespace

// CTAs of the router: one up to 512 choices (a single launch), else up to one
// per SM, 8 tokens at least in each.
int route_blocks(int64_t T, int k) {
    if (T * k <= kSingle) return 1;
    const int64_t b = (T + 7) / 8;
    return (int)(b < num_sms() ? b : num_sms());
}

cudaError_t launch_route(const void* logits, int in_f32, int64_t T, int E, int k, int score, int renorm, float scale,
                         int32_t* ids, float* weights, int32_t* offsets, int32_t* rows, int32_t* pos, int32_t* hist,
                         cudaStream_t s) {
    RouteParams p{};
    p.logits = logits;
    p.T = T;
    p.E = E;
    p.k = k;
    p.score = score;
    p.renorm = renorm;
    p.vec = E % 4 == 0 && ((uintptr_t)logits & (in_f32 ? 15 : 7)) == 0;
    p.scale = scale;
    const int ctas = route_blocks(T, k);
    p.chunk = (T + ctas - 1) / ctas;
    p.ids = ids;
    p.weights = weights;
    p.offsets = offsets;
    p.rows = rows;
    p.pos = pos;
    p.hist = hist;
    // a single CTA: a warp per token, 4 at least
    const bool eight = eight_lanes(T, E, k, ctas);
    int threads = kRouteThreads;
    if (ctas == 1) {
        const int64_t want = 32 * (T > 4 ? T : 4);
        threads = (int)(want < kRouteThreads ? want : kRouteThreads);
    }
    const size_t smem = (size_t)(2 * E + 1 + threads / 32 * E) * 4;
    const RouteKernel choose_k = in_f32 ? route_kernel<true>(E, eight) : route_kernel<false>(E, eight);
    const size_t smem_c = (size_t)E * 4 + (ctas == 1 ? kSingle * 4 + smem : 0);
    cudaError_t e = smem_c > 48 * 1024 ? set_smem_attr((const void*)choose_k, (int)smem_c) : cudaSuccess;
    if (e == cudaSuccess && smem > 48 * 1024) e = set_smem_attr((const void*)k_route_place, (int)smem);
    if (e != cudaSuccess) return e;
    e = launch_pdl(choose_k, ctas, threads, smem_c, s, p);
    if (e != cudaSuccess || ctas == 1) return e;
    return launch_pdl<RouteParams>(k_route_place, ctas, kRouteThreads, smem, s, p);
}

cudaError_t launch_combine(const void* Z, int in_f32, int64_t slots, const int32_t* pos, const float* weights, int64_t T,
                           int k, int64_t N, void* Y, int out_f32, cudaStream_t s) {
    CombineParams p{};
    p.Z = Z;
    p.slots = slots;
    p.pos = pos;
    p.weights = weights;
    p.T = T;
    p.k = k;
    p.N = N;
    p.groups = (N + 32 * kCombineCols - 1) / (32 * kCombineCols);
    p.Y = Y;
    const int64_t ctas = (T * p.groups + kCombineThreads / 32 - 1) / (kCombineThreads / 32), most = (int64_t)num_sms() * (in_f32 ? 2 : 4);
    const int64_t grid = ctas < most ? ctas : most;
    void (*kern)(const CombineParams) = in_f32 ? (out_f32 ? k_combine<true, true> : k_combine<true, false>)
                                               : (out_f32 ? k_combine<false, true> : k_combine<false, false>);
    return launch_pdl<CombineParams>(kern, grid, kCombineThreads, 0, s, p);
}

}  // namespace uw
