// uw_experts.cpp -- host entry points of the microscaled 4-bit form and of
// the expert layer: argument checks, workspace sizes, dispatch.
#include "uw_internal.h"

using namespace uw;

namespace {

bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

uw_status cuda_ok(cudaError_t e) {
    if (e == cudaSuccess) return UW_OK;
    cudaGetLastError();
    return UW_ERR_CUDA;
}

// One matrix of `rows` x K, `batch` of them.
uw_status check_matrices(int64_t batch, int64_t rows, int64_t K) {
    if (batch < 0 || rows < 0) return UW_ERR_INVALID_ARG;
    if (K < kGroup || K % kGroup || K > kMaxElems) return UW_ERR_SHAPE;
    if (rows > kMaxElems / K) return UW_ERR_SHAPE;
    if (rows && batch > kMaxElems / rows) return UW_ERR_SHAPE;
    if (rows && batch > 0x7FFFFFFF / (mx_row_tiles(rows) * mx_k_tiles(K))) return UW_ERR_SHAPE;   // one CTA per scale tile
    return UW_OK;
}

uw_status check_mx(const uw_mx_matrix* m) {
    if (!m) return UW_ERR_INVALID_ARG;
    uw_status st = check_matrices(m->batch, m->rows, m->K);
    if (st) return st;
    if (m->batch * m->rows == 0) return UW_OK;
    if (!m->codes || !m->scales || !aligned(m->codes, 32) || !aligned(m->scales, 16)) return UW_ERR_INVALID_ARG;
    return UW_OK;
}

uw_status check_weight(int64_t E, int64_t N, int64_t K) {
    if (N < 1 || K < kGroup || K % kGroup) return UW_ERR_SHAPE;
    if (N > kMaxElems / K || E > kMaxElems / N) return UW_ERR_SHAPE;
    return UW_OK;
}

uw_status check_route(int64_t T, int E, int k) {
    if (T < 0 || E < 1 || k < 1) return UW_ERR_INVALID_ARG;
    if (E > kRouteMaxE || k > kRouteMaxK || k > E || T > 0x7FFFFFFF / k) return UW_ERR_SHAPE;
    return UW_OK;
}

// One CTA needs none.
size_t route_ws_bytes(int64_t T, int E, int k) {
    const int b = T ? route_blocks(T, k) : 0;
    return b > 1 ? ((size_t)b * E * 4 + 255) & ~size_t(255) : 0;
}

uw_status check_group(const uw_group_args* a, int* src) {
    if (!a || a->slots < 0 || a->E < 1) return UW_ERR_INVALID_ARG;
    if (a->E > kRouteMaxE || a->slots > 0x7FFFFFFF - 256) return UW_ERR_SHAPE;
    const bool mx = a->W_mx || a->up_mx;
    if (mx && (a->W || a->up)) return UW_ERR_INVALID_ARG;   // one kind of weight
    *src = mx ? kGroupMx : kGroupBf16;
    return check_weight(a->E, a->N, a->K);
}

size_t group_bytes(int src, const uw_group_args* a) {
    return group_ws_bytes(src, a->slots, a->E, a->N, a->K, a->up || a->up_mx, a->rows != nullptr);
}

}  // namespace

// ===========================================================================
// microscaled 4-bit form
// ===========================================================================
extern "C" uw_status uw_mx_bytes(int64_t batch, int64_t rows, int64_t K, size_t* code_bytes, size_t* scale_bytes) {
    if (!code_bytes || !scale_bytes) return UW_ERR_INVALID_ARG;
    uw_status st = check_matrices(batch, rows, K);
    if (st) return st;
    *code_bytes = (size_t)batch * (size_t)rows * (size_t)(K / 2);
    *scale_bytes = (size_t)batch * (size_t)mx_row_tiles(rows) * (size_t)mx_k_tiles(K) * kMxTileBytes;
    return UW_OK;
}

extern "C" uw_status uw_mx_quantize(const void* X, int in_f32, int64_t batch, int64_t rows, int64_t K, uint8_t* codes,
                                    uint8_t* scales, void* stream) {
    uw_status st = check_matrices(batch, rows, K);
    if (st) return st;
    if (batch * rows == 0) return UW_OK;
    if (!X || !codes || !scales || !aligned(X, 16) || !aligned(codes, 32) || !aligned(scales, 16)) return UW_ERR_INVALID_ARG;
    return cuda_ok(launch_mx_quantize(X, in_f32, batch, rows, K, codes, scales, (cudaStream_t)stream));
}

extern "C" uw_status uw_mx_dequantize(const uw_mx_matrix* m, void* out, int out_f32, void* stream) {
    uw_status st = check_mx(m);
    if (st) return st;
    if (m->batch * m->rows == 0) return UW_OK;
    if (!out || !aligned(out, 16)) return UW_ERR_INVALID_ARG;
    return cuda_ok(launch_mx_dequantize(m->codes, m->scales, m->batch, m->rows, m->K, out, out_f32, (cudaStream_t)stream));
}

extern "C" uw_status uw_mx_gemm_workspace(int64_t M, int64_t N, int64_t K, int x_mx, size_t* bytes) {
    if (!bytes || M < 0) return UW_ERR_INVALID_ARG;
    uw_status st = check_weight(1, N, K);
    if (st) return st;
    if (M > 0x7FFFFFFF - 256) return UW_ERR_SHAPE;
    *bytes = group_ws_bytes(x_mx ? kGroupMxMx : kGroupMx, M, 1, N, K, false, false);
    return UW_OK;
}

extern "C" uw_status uw_mx_gemm(const uint16_t* X, const uw_mx_matrix* X_mx, int64_t M, const uw_mx_matrix* W, void* Y,
                                int out_f32, void* workspace, size_t workspace_bytes, void* stream) {
    if (M < 0) return UW_ERR_INVALID_ARG;
    uw_status st = check_mx(W);
    if (st) return st;
    if (W->batch != 1) return UW_ERR_SHAPE;
    size_t need = 0;
    st = uw_mx_gemm_workspace(M, W->rows, W->K, X_mx ? 1 : 0, &need);
    if (st) return st;
    if (X && X_mx) return UW_ERR_INVALID_ARG;
    if (X_mx) {
        st = check_mx(X_mx);
        if (st) return st;
        if (X_mx->batch != 1 || X_mx->rows != M || X_mx->K != W->K) return UW_ERR_SHAPE;
    }
    if (M == 0) return UW_OK;
    if ((!X && !X_mx) || !aligned(X, 16) || !Y || !aligned(Y, 16)) return UW_ERR_INVALID_ARG;
    if (!workspace || !aligned(workspace, 256) || workspace_bytes < need) return UW_ERR_WORKSPACE;
    GroupGemm g;
    g.src = X_mx ? kGroupMxMx : kGroupMx;
    g.X = X_mx ? (const void*)X_mx->codes : (const void*)X;
    g.x_scales = X_mx ? X_mx->scales : nullptr;
    g.x_rows = M;
    g.slots = M;
    g.N = W->rows;
    g.K = W->K;
    g.W = W->codes;
    g.w_scales = W->scales;
    g.Y = Y;
    g.out_f32 = out_f32 ? 1 : 0;
    g.ws = workspace;
    g.ws_bytes = workspace_bytes;
    cudaError_t e = launch_group(g, (cudaStream_t)stream, &st);
    return st ? st : cuda_ok(e);
}

// ===========================================================================
// experts
// ===========================================================================
extern "C" uw_status uw_route_workspace(int64_t T, int E, int k, size_t* bytes) {
    if (!bytes) return UW_ERR_INVALID_ARG;
    uw_status st = check_route(T, E, k);
    if (st) return st;
    *bytes = route_ws_bytes(T, E, k);
    return UW_OK;
}

extern "C" uw_status uw_route(const void* logits, int in_f32, int64_t T, int E, int k, int score, int renorm, float scale,
                              int32_t* ids, float* weights, int32_t* offsets, int32_t* rows, int32_t* pos, void* workspace,
                              size_t workspace_bytes, void* stream) {
    uw_status st = check_route(T, E, k);
    if (st) return st;
    if (score != UW_SCORE_SOFTMAX && score != UW_SCORE_SIGMOID) return UW_ERR_INVALID_ARG;
    if (!offsets || !aligned(offsets, 4)) return UW_ERR_INVALID_ARG;
    if (T == 0) return cuda_ok(cudaMemsetAsync(offsets, 0, (size_t)(E + 1) * 4, (cudaStream_t)stream));
    if (!logits || !ids || !weights || !rows || !pos) return UW_ERR_INVALID_ARG;
    if (!aligned(logits, in_f32 ? 4 : 2) || !aligned(ids, 4) || !aligned(weights, 4) || !aligned(rows, 4) || !aligned(pos, 4))
        return UW_ERR_INVALID_ARG;
    const size_t need = route_ws_bytes(T, E, k);
    if (need && (!workspace || !aligned(workspace, 256) || workspace_bytes < need)) return UW_ERR_WORKSPACE;
    return cuda_ok(launch_route(logits, in_f32, T, E, k, score, renorm ? 1 : 0, scale, ids, weights, offsets, rows, pos,
                                (int32_t*)workspace, (cudaStream_t)stream));
}

extern "C" uw_status uw_gemm_grouped_workspace(const uw_group_args* a, size_t* bytes) {
    if (!bytes) return UW_ERR_INVALID_ARG;
    int src;
    uw_status st = check_group(a, &src);
    if (st) return st;
    *bytes = group_bytes(src, a);
    return UW_OK;
}

extern "C" uw_status uw_gemm_grouped(const uw_group_args* a, void* stream) {
    int src;
    uw_status st = check_group(a, &src);
    if (st) return st;
    if (src == kGroupMx) {
        const uw_mx_matrix* w[2] = {a->W_mx, a->up_mx};
        for (int i = 0; i < 2; i++) {
            if (i && !w[i]) break;
            st = check_mx(w[i]);
            if (st) return st;
            if (w[i]->batch != a->E || w[i]->rows != a->N || w[i]->K != a->K) return UW_ERR_SHAPE;
        }
    } else if (!a->W || !aligned(a->W, 16) || !aligned(a->up, 16)) {
        return UW_ERR_INVALID_ARG;
    }
    if (a->slots == 0) return UW_OK;
    if (!a->X || !aligned(a->X, 16) || !a->Y || !aligned(a->Y, 16)) return UW_ERR_INVALID_ARG;
    if (!a->offsets || !aligned(a->offsets, 4) || !aligned(a->rows, 4)) return UW_ERR_INVALID_ARG;
    if (a->x_rows < 1 || (!a->rows && a->x_rows < a->slots)) return UW_ERR_INVALID_ARG;
    if (a->x_rows > 0x7FFFFFFF - 256) return UW_ERR_SHAPE;
    if (!a->workspace || !aligned(a->workspace, 256) || a->workspace_bytes < group_bytes(src, a))
        return UW_ERR_WORKSPACE;
    GroupGemm g;
    g.src = src;
    g.X = a->X;
    g.x_rows = a->x_rows;
    g.rows = a->rows;
    g.slots = a->slots;
    g.offsets = a->offsets;
    g.E = a->E;
    g.N = a->N;
    g.K = a->K;
    g.W = src == kGroupMx ? (const void*)a->W_mx->codes : (const void*)a->W;
    g.up = src == kGroupMx ? (a->up_mx ? (const void*)a->up_mx->codes : nullptr) : (const void*)a->up;
    if (src == kGroupMx) {
        g.w_scales = a->W_mx->scales;
        g.up_scales = a->up_mx ? a->up_mx->scales : nullptr;
    }
    g.Y = a->Y;
    g.out_f32 = a->out_f32 ? 1 : 0;
    g.ws = a->workspace;
    g.ws_bytes = a->workspace_bytes;
    cudaError_t e = launch_group(g, (cudaStream_t)stream, &st);
    return st ? st : cuda_ok(e);
}

extern "C" uw_status uw_combine(const void* Z, int in_f32, int64_t slots, const int32_t* pos, const float* weights, int64_t T,
                                int k, int64_t N, void* Y, int out_f32, void* stream) {
    if (slots < 0 || T < 0 || k < 1 || N < 0) return UW_ERR_INVALID_ARG;
    if (k > kRouteMaxK || T > 0x7FFFFFFF / k) return UW_ERR_SHAPE;
    if (N > 0x7FFFFFFF || (T && (N + 7) / 8 > (int64_t)0x7FFFFFFF * 256 / T)) return UW_ERR_SHAPE;
    if (T == 0 || N == 0) return UW_OK;
    if (!pos || !weights || !Y || (slots && !Z)) return UW_ERR_INVALID_ARG;
    if (!aligned(Z, 16) || !aligned(Y, 16) || !aligned(pos, 4) || !aligned(weights, 4)) return UW_ERR_INVALID_ARG;
    return cuda_ok(launch_combine(Z, in_f32, slots, pos, weights, T, k, N, Y, out_f32, (cudaStream_t)stream));
}
