// uw_route.cu -- the ends of an expert layer: the router's choice with the
// slots sorted by expert, and the weighted sum of the experts' outputs.
//
// Router.  The choice compares logits only (softmax and sigmoid rise with
// the logit), by an order-preserving 32-bit key, so it is exact whatever the
// scores round to.  A warp owns a token: E/32 keys a lane, k rounds of one
// warp-wide maximum and one minimum over the indices that reach it.  Scores
// are fp32 with the accurate exponential.
// Slots.  A stable counting sort over at most one CTA per SM: CTA b owns a
// contiguous run of tokens, counts its choices per expert (k_route_choose),
// and after all counts are known (k_route_place) adds up the counts of the
// CTAs before it, the experts before each expert and, inside the CTA, of the
// warps before each warp.  Ranks inside a warp come from match_any, so the
// order -- and every output -- is the same on every run.  What bounds it: the
// logits are read once; below a few thousand tokens the launches' latency.
// With few choices one CTA does both parts in a single launch.
//
// Combination.  Y[t] = sum_j w[t,j] Z[pos[t,j]]: bound by reading T k N and
// writing T N values once; a thread owns 8 columns of one token and has its
// first eight choices' rows in flight before it adds.
#include "uw_device.cuh"
#include "uw_internal.h"

namespace uw {

int route_status_take() { return unit_status_take(); }

namespace {

constexpr int kRouteThreads = 1024;   // at most; a single CTA takes a warp per token
constexpr uint32_t kFull = 0xFFFFFFFFu;
constexpr int kSingle = 512;     // choices up to which one CTA does everything

struct RouteParams {
    const void* logits;
    int64_t T;
    int E, k, score, renorm;
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

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(kFull, v, d);
    return v;
}

// Logits of token t, expert 32 i + lane, as fp32 bits (NaN past E); all loads
// are issued before any is used.
template <int VPL, bool F32>
__device__ __forceinline__ void load_logits(const RouteParams& p, int64_t t, int lane, uint32_t (&raw)[VPL]) {
    if (F32) {
        const uint32_t* x = reinterpret_cast<const uint32_t*>(p.logits) + t * p.E + lane;
#pragma unroll
        for (int i = 0; i < VPL; i++) raw[i] = 32 * i + lane < p.E ? __ldg(x + 32 * i) : 0x7FC00000u;
    } else {
        const uint16_t* x = reinterpret_cast<const uint16_t*>(p.logits) + t * p.E + lane;
#pragma unroll
        for (int i = 0; i < VPL; i++) raw[i] = 32 * i + lane < p.E ? (uint32_t)__ldg(x + 32 * i) : 0x7FC0u;
#pragma unroll
        for (int i = 0; i < VPL; i++) raw[i] <<= 16;
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

// The k largest keys in falling order, equal keys by index: lane j < k ends up
// with choice j.  k rounds of a maximum over the warp and a minimum over the
// indices that reach it.
template <int VPL>
__device__ __noinline__ uint2 select_exact(const RouteParams& p, int64_t t, int lane) {
    uint32_t key[VPL];
    load_logits<VPL, true>(p, t, lane, key);
#pragma unroll
    for (int i = 0; i < VPL; i++) key[i] = bits_key(key[i]);
    uint2 mine = make_uint2(0xFFFFFFFFu, 0);   // (expert, key)
    for (int j = 0; j < p.k; j++) {
        uint32_t best = 0, cand = 0xFFFFFFFFu;
#pragma unroll
        for (int i = 0; i < VPL; i++) best = best > key[i] ? best : key[i];
        const uint32_t mx = __reduce_max_sync(kFull, best);
        if (mx == 0) break;
#pragma unroll
        for (int i = VPL - 1; i >= 0; i--)
            if (key[i] == mx) cand = (uint32_t)(32 * i + lane);
        const uint32_t e = __reduce_min_sync(kFull, cand);
#pragma unroll
        for (int i = 0; i < VPL; i++)
            if ((uint32_t)(32 * i + lane) == e) key[i] = 0;
        if (lane == j) mine = make_uint2(e, mx);
    }
    return mine;
}

// One token: lane j < k ends up with choice j (expert id, or -1) and weight.
// The rounds run on words that join a key's upper 22 bits with the index: one
// maximum a round, and the word that gave it is unique.  Where two
// neighbours of the k + 1 largest share those 22 bits and fp32 logits may
// differ below them (about 1 token in 50), the selection is repeated exactly;
// the upper 22 bits hold all of a BF16 logit.
template <int VPL, bool F32>
__device__ __forceinline__ void choose(const RouteParams& p, int64_t t, const uint32_t (&raw)[VPL], int lane, int& id,
                                       float& w) {
    uint32_t word[VPL];
    uint32_t best = 0;
    float total = 0.0f, m = 0.0f;
#pragma unroll
    for (int i = 0; i < VPL; i++) word[i] = bits_key(raw[i]);
    if (p.score == UW_SCORE_SOFTMAX) {
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < VPL; i++) top = top > word[i] ? top : word[i];
        top = __reduce_max_sync(kFull, top);
        m = key_logit(top);   // top = 0 (no choice at all): unused
        if (!p.renorm && top) {   // the denominator over every logit
#pragma unroll
            for (int i = 0; i < VPL; i++)
                if (word[i]) total += expf(key_logit(word[i]) - m);
            total = warp_sum(total);
        }
    }
#pragma unroll
    for (int i = 0; i < VPL; i++) {
        word[i] = word[i] ? (word[i] & 0xFFFFFC00u) | (uint32_t)(1023 - (32 * i + lane)) : 0u;
        best = best > word[i] ? best : word[i];
    }
    uint32_t got = 0;
    const int rounds = F32 && p.k < 32 ? p.k + 1 : p.k;   // one more: does the last choice stand out
    for (int j = 0; j < rounds; j++) {
        const uint32_t mx = __reduce_max_sync(kFull, best);
        if (mx == 0) break;
        if (lane == j) got = mx;
        // the largest word below mx: word - mx wraps to the top of the range below it, to its bottom from it up
        uint32_t below = 0;
#pragma unroll
        for (int i = 0; i < VPL; i++) below = __viaddmax_u32(word[i], 0u - mx, below);
        best = below + mx;
        best = best < mx ? best : 0u;
    }
    id = got && lane < p.k ? 1023 - (int)(got & 1023u) : -1;
    uint32_t mine = 0;
    bool close = false;
    if (F32) {
        const uint32_t before = __shfl_up_sync(kFull, got, 1);
        close = lane && got && (before >> 10) == (got >> 10);
        // k = 32 has no extra round: what is left over is compared with the last choice
        const uint32_t last = __shfl_sync(kFull, got, 31);
        if (p.k == 32) close |= best && (best >> 10) == (last >> 10);
    }
    if (F32 && __any_sync(kFull, close)) {
        const uint2 x = select_exact<VPL>(p, t, lane);
        id = (int)x.x;
        mine = x.y;
    } else if (id >= 0) {
        mine = F32 ? bits_key(__ldg(reinterpret_cast<const uint32_t*>(p.logits) + t * p.E + id)) : got & 0xFFFFFC00u;
    }
    if (!F32 && mine) mine |= mine >> 31 ? 0u : 0x3FFu;   // a negative logit's key has its low bits set
    const float x = key_logit(mine);
    float s = 0.0f;
    if (mine) s = p.score == UW_SCORE_SOFTMAX ? expf(x - m) : 1.0f / (1.0f + expf(-x));
    if (p.renorm) total = warp_sum(s);
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

template <int VPL, bool F32>
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
    uint32_t raw[VPL], next[VPL];
    if (t0 + warp < t1) load_logits<VPL, F32>(p, t0 + warp, lane, next);
    for (int64_t t = t0 + warp; t < t1; t += warps) {
#pragma unroll
        for (int i = 0; i < VPL; i++) raw[i] = next[i];
        if (t + warps < t1) load_logits<VPL, F32>(p, t + warps, lane, next);   // the next token's, meanwhile
        int id;
        float w;
        choose<VPL, F32>(p, t, raw, lane, id, w);
        if (lane < p.k) {
            p.ids[t * p.k + lane] = id;
            p.weights[t * p.k + lane] = w;
            if (id >= 0) atomicAdd(&counts[id], 1);
            if (single) ids[t * p.k + lane] = id;
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
template <bool F32>
RouteKernel route_kernel(int E) {
    return E <= 32    ? k_route_choose<1, F32>
           : E <= 64  ? k_route_choose<2, F32>
           : E <= 128 ? k_route_choose<4, F32>
           : E <= 256 ? k_route_choose<8, F32>
           : E <= 512 ? k_route_choose<16, F32>
                      : k_route_choose<32, F32>;
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
    int64_t groups;   // column groups of 8
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
    const int64_t i = (int64_t)blockIdx.x * kCombineThreads + threadIdx.x;
    if (i >= p.T * p.groups) return;
    const int64_t t = i / p.groups, c = (i - t * p.groups) * kCombineCols;
    const bool vec = p.N % 8 == 0;
    const int n = p.N - c < 8 ? (int)(p.N - c) : 8;
    float acc[8] = {};
    for (int j0 = 0; j0 < p.k; j0 += kCombineAhead) {
        // all positions, then all rows: nothing in between that the loads would wait for
        Cols<IN32> z[kCombineAhead];
        float w[kCombineAhead];
        int32_t s[kCombineAhead];
#pragma unroll
        for (int j = 0; j < kCombineAhead; j++) {
            s[j] = j0 + j < p.k ? __ldg(p.pos + t * p.k + j0 + j) : -1;
            w[j] = j0 + j < p.k ? __ldg(p.weights + t * p.k + j0 + j) : 0.0f;
        }
#pragma unroll
        for (int j = 0; j < kCombineAhead; j++) {
            z[j].a = z[j].b = make_uint4(0, 0, 0, 0);
            if (s[j] >= 0 && s[j] < p.slots) load_cols<IN32>(p.Z, s[j] * p.N + c, n, vec, z[j]);
        }
        bool wrong = false;
#pragma unroll
        for (int j = 0; j < kCombineAhead; j++) {
            wrong |= s[j] >= p.slots;
            add_cols<IN32>(z[j], s[j] < 0 || s[j] >= p.slots ? 0.0f : w[j], acc);
        }
        if (wrong) raise_status(UW_ERR_DEVICE);
    }
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
    int threads = kRouteThreads;
    if (ctas == 1) {
        const int64_t want = 32 * (T > 4 ? T : 4);
        threads = (int)(want < kRouteThreads ? want : kRouteThreads);
    }
    const size_t smem = (size_t)(2 * E + 1 + threads / 32 * E) * 4;
    const RouteKernel choose_k = in_f32 ? route_kernel<true>(E) : route_kernel<false>(E);
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
    p.groups = (N + kCombineCols - 1) / kCombineCols;
    p.Y = Y;
    const int64_t grid = (T * p.groups + kCombineThreads - 1) / kCombineThreads;
    void (*kern)(const CombineParams) = in_f32 ? (out_f32 ? k_combine<true, true> : k_combine<true, false>)
                                               : (out_f32 ? k_combine<false, true> : k_combine<false, false>);
    return launch_pdl<CombineParams>(kern, grid, kCombineThreads, 0, s, p);
}

}  // namespace uw
