// uw_mx.cu -- the microscaled 4-bit form (MXFP4): quantisation of BF16 or
// fp32 matrices to e2m1 codes with one e8m0 scale per 32 values of a row, and
// the way back.  The byte layout is stated in unweight.h.
//
// Mathematics: with a the block's largest magnitude, s = floor(log2 a) - 2
// puts a / 2^s into [4, 8), so the block uses the format's largest binade
// (values 4 and 6; what rounds above 6 saturates).  floor(log2 a) is a's
// exponent field, and dividing by 2^s is exact in fp32, so each value is
// rounded once, by the conversion instruction (nearest, ties to even).
//
// Both kernels are bound by HBM: they read and write every byte once.  A CTA
// owns one scale tile (128 rows x 256 k): a warp's step is one row of the
// tile, 8 values a lane (a 16-byte load of BF16), four lanes a block, and the
// tile's 1024 scale bytes are gathered in shared memory and leave as one
// contiguous run.  The CTA's rows are loaded eight steps ahead of their use.
// Measured: 14336 x 4096 from fp32 and back to BF16 in 77 us for both, 5.4 TB/s
// (the copy bandwidth is 6.5); 37 x 4096 from BF16 and back in 4.6 us, two
// launches' latency.
#include <cuda_fp16.h>

#include "uw_device.cuh"
#include "uw_internal.h"

namespace uw {
namespace {

constexpr int kMxThreads = 256;
constexpr int kMxWarps = kMxThreads / 32;
constexpr int kMxAhead = 8;   // rows a warp has in flight

// 8 fp32 magnitudes -> 8 codes (value i in bits 4i..4i+3).
__device__ __forceinline__ uint32_t to_codes(const float (&v)[8]) {
    uint32_t d;
    asm("{\n\t.reg .b8 a, b, c, e;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 e, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, e};\n\t}"
        : "=r"(d)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return d;
}

template <bool F32>
struct Row8 {
    uint4 a, b;   // b: fp32 only
};

template <bool F32>
__device__ __forceinline__ Row8<F32> load8(const void* X, int64_t i) {
    Row8<F32> r;
    if (F32) {
        const uint4* p = reinterpret_cast<const uint4*>(reinterpret_cast<const float*>(X) + i);
        r.a = __ldcs(p);
        r.b = __ldcs(p + 1);
    } else {
        r.a = __ldcs(reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(X) + i));
    }
    return r;
}

template <bool F32>
__device__ __forceinline__ void widen8(const Row8<F32>& r, float (&v)[8]) {
    const uint32_t a[4] = {r.a.x, r.a.y, r.a.z, r.a.w};
    if (F32) {
        const uint32_t b[4] = {r.b.x, r.b.y, r.b.z, r.b.w};
#pragma unroll
        for (int i = 0; i < 4; i++) {
            v[i] = __uint_as_float(a[i]);
            v[4 + i] = __uint_as_float(b[i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; i++) {
            v[2 * i] = __uint_as_float(a[i] << 16);
            v[2 * i + 1] = __uint_as_float(a[i] & 0xFFFF0000u);
        }
    }
}

template <bool F32>
__global__ void __launch_bounds__(kMxThreads)
    k_mx_quantize(const void* __restrict__ X, int64_t rows, int64_t K, int row_tiles, int k_tiles,
                  uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
    __shared__ uint32_t tile[kMxTileBytes / 4];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t t = blockIdx.x;
    const int kt = (int)(t % k_tiles);
    const int64_t m = t / k_tiles;                        // (matrix, row tile)
    const int64_t r0 = (m % row_tiles) * kMxTileRows, mat = m / row_tiles;
    const int64_t k = (int64_t)kt * kMxTileK + 8 * lane;
    tile[threadIdx.x] = 0;   // bytes of rows and blocks past the matrix
    __syncthreads();
    uint8_t* tb = reinterpret_cast<uint8_t*>(tile);
    const int nr = rows - r0 < kMxTileRows ? (int)(rows - r0) : kMxTileRows;
    const bool in_k = k < K;   // K is a multiple of 64: a block's four lanes agree
    const int64_t base = (mat * rows + r0) * K + k;
    const int b = lane >> 2;
    const int sb = ((b >> 2) << 9) + (b & 3);             // byte of this block in its rows' 16-byte groups
    for (int rr = warp; rr < nr; rr += kMxWarps * kMxAhead) {
        Row8<F32> in[kMxAhead];
#pragma unroll
        for (int i = 0; i < kMxAhead; i++) {
            const int r = rr + i * kMxWarps;
            if (r < nr && in_k) in[i] = load8<F32>(X, base + (int64_t)r * K);
        }
#pragma unroll
        for (int i = 0; i < kMxAhead; i++) {
            const int r = rr + i * kMxWarps;
            if (r >= nr) break;
            float v[8];
            if (in_k) {
                widen8<F32>(in[i], v);
            } else {
#pragma unroll
                for (int q = 0; q < 8; q++) v[q] = 0.0f;
            }
            // largest magnitude of the block, by its bits (NaN and infinity sort above every number)
            uint32_t a = 0;
#pragma unroll
            for (int q = 0; q < 8; q++) {
                const uint32_t x = __float_as_uint(v[q]) & 0x7FFFFFFFu;
                a = a > x ? a : x;
            }
            uint32_t o = __shfl_xor_sync(0xFFFFFFFFu, a, 1);
            a = a > o ? a : o;
            o = __shfl_xor_sync(0xFFFFFFFFu, a, 2);
            a = a > o ? a : o;
            const uint32_t e = a >> 23;                   // floor(log2 a) + 127
            const bool bad = e == 255u;
            const uint32_t sbyte = bad ? 255u : (e > 2u ? e - 2u : 0u);
            const float inv = __uint_as_float((254u - (bad ? 0u : sbyte)) << 23);   // 2^-s, s in [-127, 125]
#pragma unroll
            for (int q = 0; q < 8; q++) v[q] = bad ? 0.0f : v[q] * inv;
            if (in_k) {
                const uint32_t c = to_codes(v);
                __stcs(reinterpret_cast<uint32_t*>(codes + ((base + (int64_t)r * K) >> 1)), c);
                if ((lane & 3) == 0) tb[sb + ((r & 31) << 4) + ((r >> 5) << 2)] = (uint8_t)sbyte;
            }
        }
    }
    __syncthreads();
    reinterpret_cast<uint32_t*>(scales)[t * (kMxTileBytes / 4) + threadIdx.x] = tile[threadIdx.x];
}

// 8 codes -> 8 magnitudes with sign, as fp32.
__device__ __forceinline__ void from_codes(uint32_t c, float (&v)[8]) {
    uint32_t h[4];
    asm("{\n\t.reg .b8 a, b, c, e;\n\t"
        "mov.b32 {a, b, c, e}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, e;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(c));
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const __half2 x = *reinterpret_cast<const __half2*>(&h[i]);
        v[2 * i] = __low2float(x);
        v[2 * i + 1] = __high2float(x);
    }
}

template <bool F32>
__global__ void __launch_bounds__(kMxThreads)
    k_mx_dequantize(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales, int64_t rows, int64_t K,
                    int row_tiles, int k_tiles, void* __restrict__ out) {
    __shared__ uint32_t tile[kMxTileBytes / 4];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t t = blockIdx.x;
    const int kt = (int)(t % k_tiles);
    const int64_t m = t / k_tiles;
    const int64_t r0 = (m % row_tiles) * kMxTileRows, mat = m / row_tiles;
    const int64_t k = (int64_t)kt * kMxTileK + 8 * lane;
    tile[threadIdx.x] = reinterpret_cast<const uint32_t*>(scales)[t * (kMxTileBytes / 4) + threadIdx.x];
    __syncthreads();
    const uint8_t* tb = reinterpret_cast<const uint8_t*>(tile);
    const int nr = rows - r0 < kMxTileRows ? (int)(rows - r0) : kMxTileRows;
    if (k >= K) return;
    const int64_t base = (mat * rows + r0) * K + k;
    const int b = lane >> 2;
    const int sb = ((b >> 2) << 9) + (b & 3);
    for (int rr = warp; rr < nr; rr += kMxWarps * kMxAhead) {
        uint32_t in[kMxAhead];
#pragma unroll
        for (int i = 0; i < kMxAhead; i++) {
            const int r = rr + i * kMxWarps;
            if (r < nr) in[i] = __ldcs(reinterpret_cast<const uint32_t*>(codes + ((base + (int64_t)r * K) >> 1)));
        }
#pragma unroll
        for (int i = 0; i < kMxAhead; i++) {
            const int r = rr + i * kMxWarps;
            if (r >= nr) break;
            const uint32_t s = tb[sb + ((r & 31) << 4) + ((r >> 5) << 2)];
            // 2^s: an exponent field, the subnormal 2^-127, or NaN
            const float f = __uint_as_float(s == 255u ? 0x7FC00000u : s ? s << 23 : 0x00400000u);
            float v[8];
            from_codes(in[i], v);
#pragma unroll
            for (int q = 0; q < 8; q++) v[q] *= f;
            const int64_t at = base + (int64_t)r * K;
            if (F32) {
                float4* p = reinterpret_cast<float4*>(reinterpret_cast<float*>(out) + at);
                __stcs(p, make_float4(v[0], v[1], v[2], v[3]));
                __stcs(p + 1, make_float4(v[4], v[5], v[6], v[7]));
            } else {
                uint4 w;
                uint32_t* wp = &w.x;
#pragma unroll
                for (int q = 0; q < 4; q++) {
                    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * q], v[2 * q + 1]);
                    wp[q] = *reinterpret_cast<const uint32_t*>(&h);
                }
                __stcs(reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(out) + at), w);
            }
        }
    }
}

template <typename... P, typename... A>
cudaError_t launch_tiles(void (*kern)(P...), int64_t tiles, cudaStream_t s, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)tiles);
    cfg.blockDim = dim3(kMxThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, kern, P(args)...);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_mx_quantize(const void* X, int in_f32, int64_t batch, int64_t rows, int64_t K, uint8_t* codes,
                               uint8_t* scales, cudaStream_t s) {
    const int64_t rt = mx_row_tiles(rows), kt = mx_k_tiles(K);
    return launch_tiles(in_f32 ? k_mx_quantize<true> : k_mx_quantize<false>, batch * rt * kt, s, X, rows, K, (int)rt, (int)kt,
                        codes, scales);
}

cudaError_t launch_mx_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t batch, int64_t rows, int64_t K,
                                 void* out, int out_f32, cudaStream_t s) {
    const int64_t rt = mx_row_tiles(rows), kt = mx_k_tiles(K);
    return launch_tiles(out_f32 ? k_mx_dequantize<true> : k_mx_dequantize<false>, batch * rt * kt, s, codes, scales, rows, K,
                        (int)rt, (int)kt, out);
}

}  // namespace uw
