// C-ABI entry points of the recurrent layer's operators around the KDA kernels (declared in
// include/kda.h): argument validation on the host, then launches on the caller's stream.
#include <math.h>

#include "kda_common.cuh"
#include "kda_layer.h"

namespace {

constexpr int kMostChannels = 1 << 20;

bool dtype_ok(kda_dtype d) { return d == KDA_F32 || d == KDA_BF16; }
size_t size_of(kda_dtype d) { return d == KDA_BF16 ? 2 : 4; }
kda_status from_cuda(cudaError_t e) { return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA; }
bool aligned(const void* p, size_t to) { return (uintptr_t)p % to == 0; }

struct Span {
    const void* p;
    size_t n;
};
Span rows(const void* p, int64_t count, int64_t ld, int64_t width, size_t es) {
    return {p, count > 0 ? (size_t)((count - 1) * ld + width) * es : 0};
}
bool overlap(const Span& a, const Span& b) {
    const char* x = static_cast<const char*>(a.p);
    const char* y = static_cast<const char*>(b.p);
    return x && y && a.n && b.n && x < y + b.n && y < x + a.n;
}
// No output overlaps an input or another output.
template <int NI, int NO>
bool apart(const Span (&in)[NI], const Span (&out)[NO]) {
    for (int o = 0; o < NO; ++o) {
        for (int i = 0; i < NI; ++i)
            if (overlap(out[o], in[i])) return false;
        for (int q = o + 1; q < NO; ++q)
            if (overlap(out[o], out[q])) return false;
    }
    return true;
}

// Pages and list entries of the pages calls, rows of the single-token ones: they are counted in 32 bits.
constexpr int kMostPages = 1 << 30, kMostRows = 1 << 30;

kda_status clear(int32_t* status, cudaStream_t st) {
    if (status && cudaMemsetAsync(status, 0, sizeof(int32_t), st) != cudaSuccess) return KDA_ERR_CUDA;
    return KDA_OK;
}

// Tokens, sequences and channels of a packed or dense call.
kda_status check_stream(int B, int T, int C, int N, const int32_t* cu) {
    if (B < 0 || T < 0 || C <= 0 || N < 0) return KDA_ERR_INVALID_ARG;
    // (kernels step past their ends by up to a grid's blocks or a tile)
    if ((int64_t)B * T > 0x7fffffffLL - 65536 || N > 0x7fffffff - 65536) return KDA_ERR_INVALID_ARG;
    if (cu ? B != 1 : N != B) return KDA_ERR_INVALID_ARG;
    if (!aligned(cu, 4)) return KDA_ERR_INVALID_ARG;
    if (C > kMostChannels) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

kda_status check_conv(int64_t ldx, const float* weight, const float* bias, int C, int W, int act) {
    if (W < 2 || W > 4) return KDA_ERR_UNSUPPORTED;
    if (ldx < C || !weight || !aligned(weight, 4) || !aligned(bias, 4) || (act != 0 && act != 1)) return KDA_ERR_INVALID_ARG;
    return KDA_OK;
}

// Tokens of a scan's backward pass: 65535 chunks of 64.
constexpr int kMostBwdTokens = 65535 * 64;
// Stands for offsets where only their presence matters.
const int32_t* const kPacked = reinterpret_cast<const int32_t*>(16);

kda_status scan_sizes(kda::SsmScanParams& p, int B, int T, int C, int G, int S, int N, const int32_t* cu) {
    const kda_status s = check_stream(B, T, C, N, cu);
    if (s != KDA_OK) return s;
    if (G <= 0 || C % G != 0) return KDA_ERR_INVALID_ARG;
    if (S != 8 && S != 16 && S != 32 && S != 64) return KDA_ERR_UNSUPPORTED;
    p.cu = cu; p.T = T; p.N = N; p.C = C; p.G = G; p.S = S; p.total = B * T;
    return KDA_OK;
}

// The inputs that the forward and backward scans share.
kda_status scan_inputs(const kda::SsmScanParams& p, kda_dtype dtype) {
    if (!dtype_ok(dtype)) return KDA_ERR_UNSUPPORTED;
    if (p.softplus != 0 && p.softplus != 1) return KDA_ERR_INVALID_ARG;
    const int64_t vec = (int64_t)p.G * p.S;
    if (p.ldu < p.C || p.ldd < p.C || (p.z && p.ldz < p.C) || p.ldb < vec || p.ldc < vec) return KDA_ERR_INVALID_ARG;
    if (!p.A || (p.total > 0 && (!p.u || !p.delta || !p.Bm || !p.Cm))) return KDA_ERR_INVALID_ARG;
    for (const void* q : {p.u, p.delta, p.Bm, p.Cm, p.z})
        if (!aligned(q, size_of(dtype))) return KDA_ERR_INVALID_ARG;
    if (!kda_host::aligned16(p.A) || !kda_host::aligned16(p.initial)) return KDA_ERR_INVALID_ARG;
    if (!aligned(p.D, 4) || !aligned(p.bias, 4)) return KDA_ERR_INVALID_ARG;
    return KDA_OK;
}
#define SCAN_INPUT_SPANS(in, p, es)                                                                                       \
    const Span in[] = {rows(p.u, p.total, p.ldu, p.C, es), rows(p.delta, p.total, p.ldd, p.C, es),                        \
                       rows(p.z, p.total, p.ldz, p.C, es), rows(p.Bm, p.total, p.ldb, (int64_t)p.G * p.S, es),            \
                       rows(p.Cm, p.total, p.ldc, (int64_t)p.G * p.S, es), {p.A, (size_t)p.C * p.S * 4},                  \
                       {p.D, (size_t)p.C * 4}, {p.bias, (size_t)p.C * 4}, {p.initial, (size_t)p.N * p.C * p.S * 4},       \
                       {p.cu, (size_t)(p.N + 1) * 4}}

}  // namespace

extern "C" {

kda_status kda_short_conv_fwd(const void* x, int64_t ldx, const float* weight, const float* bias, int conv_act,
                              kda_dtype dtype, const void* initial, const int32_t* cu_seqlens, int B, int T, int C,
                              int W, int N, void* y, void* final_history, void* stream) {
    kda_status s = check_stream(B, T, C, N, cu_seqlens);
    if (s != KDA_OK) return s;
    if (!dtype_ok(dtype)) return KDA_ERR_UNSUPPORTED;
    if ((s = check_conv(ldx, weight, bias, C, W, conv_act)) != KDA_OK) return s;
    const int64_t total = (int64_t)B * T;
    const size_t es = size_of(dtype);
    if (total > 0 && (!x || !y)) return KDA_ERR_INVALID_ARG;
    for (const void* p : {x, (const void*)y, initial, (const void*)final_history})
        if (!aligned(p, es)) return KDA_ERR_INVALID_ARG;
    const size_t hist = (size_t)N * (W - 1) * C * es;
    const Span in[] = {rows(x, total, ldx, C, es), {weight, (size_t)C * W * 4}, {bias, (size_t)C * 4}, {initial, hist},
                       {cu_seqlens, (size_t)(N + 1) * 4}};
    const Span out[] = {{y, (size_t)total * C * es}, {final_history, hist}};
    if (!apart(in, out)) return KDA_ERR_INVALID_ARG;
    if (N == 0) return KDA_OK;
    kda::ConvParams p{};
    p.x = x; p.ldx = ldx; p.weight = weight; p.bias = bias; p.act = conv_act;
    p.initial = initial; p.cu = cu_seqlens; p.T = T; p.N = N; p.C = C; p.W = W; p.total = (int)total;
    p.y = y; p.final_hist = final_history;
    return from_cuda(kda::short_conv_fwd(dtype, p, (cudaStream_t)stream));
}

size_t kda_short_conv_bwd_workspace_size(int B, int T, int C, int W) {
    if (check_stream(B, T, C, B, nullptr) != KDA_OK || W < 2 || W > 4) return 0;
    return kda::short_conv_bwd_partial(B * T, C, W) * sizeof(float);
}

kda_status kda_short_conv_bwd(const void* x, int64_t ldx, const float* weight, const float* bias, int conv_act,
                              kda_dtype dtype, const void* initial, const int32_t* cu_seqlens, int B, int T, int C,
                              int W, int N, const void* dy, const void* dfinal, kda_dtype grad_dtype, void* dx,
                              float* dweight, float* dbias, void* dinitial, void* workspace, size_t workspace_bytes,
                              void* stream) {
    kda_status s = check_stream(B, T, C, N, cu_seqlens);
    if (s != KDA_OK) return s;
    if (!dtype_ok(dtype) || !dtype_ok(grad_dtype) || (dtype == KDA_F32 && grad_dtype != KDA_F32)) return KDA_ERR_UNSUPPORTED;
    if ((s = check_conv(ldx, weight, bias, C, W, conv_act)) != KDA_OK) return s;
    const int64_t total = (int64_t)B * T;
    const size_t es = size_of(dtype), gs = size_of(grad_dtype);
    if (!dweight || (total > 0 && (!x || !dy || !dx))) return KDA_ERR_INVALID_ARG;
    for (const void* p : {x, initial})
        if (!aligned(p, es)) return KDA_ERR_INVALID_ARG;
    for (const void* p : {dy, dfinal, (const void*)dx, (const void*)dinitial})
        if (!aligned(p, gs)) return KDA_ERR_INVALID_ARG;
    if (!aligned(dweight, 4) || !aligned(dbias, 4)) return KDA_ERR_INVALID_ARG;
    const size_t need = kda::short_conv_bwd_partial((int)total, C, W) * sizeof(float);
    if (workspace_bytes < need || !workspace) return KDA_ERR_WORKSPACE;
    if (!kda_host::aligned16(workspace)) return KDA_ERR_INVALID_ARG;
    const size_t hist = (size_t)N * (W - 1) * C;
    const Span in[] = {rows(x, total, ldx, C, es), {weight, (size_t)C * W * 4}, {bias, (size_t)C * 4}, {initial, hist * es},
                       {cu_seqlens, (size_t)(N + 1) * 4}, {dy, (size_t)total * C * gs}, {dfinal, hist * gs}};
    const Span out[] = {{dx, (size_t)total * C * gs}, {dweight, (size_t)C * W * 4}, {dbias, (size_t)C * 4},
                        {dinitial, hist * gs}, {workspace, need}};
    if (!apart(in, out)) return KDA_ERR_INVALID_ARG;
    kda::ConvParams p{};
    p.x = x; p.ldx = ldx; p.weight = weight; p.bias = bias; p.act = conv_act;
    p.initial = initial; p.cu = cu_seqlens; p.T = T; p.N = N; p.C = C; p.W = W; p.total = (int)total;
    p.dy = dy; p.dfinal = dfinal; p.dx = dx; p.dinitial = dinitial; p.dweight = dweight; p.dbias = dbias;
    p.partial = static_cast<float*>(workspace);
    return from_cuda(kda::short_conv_bwd(dtype, grad_dtype, p, (cudaStream_t)stream));
}

kda_status kda_short_conv_step(const void* x, int64_t ldx, const float* weight, const float* bias, int conv_act,
                               kda_dtype dtype, void* history, const int32_t* slots, int P, int N, int C, int W,
                               void* y, int32_t* status, void* stream) {
    if (N < 0 || P < 0 || C <= 0) return KDA_ERR_INVALID_ARG;
    if (!dtype_ok(dtype) || C > kMostChannels || N > kMostRows || (slots && N > KDA_MOST_SLOTS)) return KDA_ERR_UNSUPPORTED;
    const kda_status s = check_conv(ldx, weight, bias, C, W, conv_act);
    if (s != KDA_OK) return s;
    const size_t es = size_of(dtype);
    if (N > 0 && (!x || !history || !y || P == 0)) return KDA_ERR_INVALID_ARG;
    if (!slots && N > P) return KDA_ERR_INVALID_ARG;
    for (const void* p : {x, (const void*)history, (const void*)y})
        if (!aligned(p, es)) return KDA_ERR_INVALID_ARG;
    if (!aligned(slots, 4) || !aligned(status, 4)) return KDA_ERR_INVALID_ARG;
    const Span in[] = {rows(x, N, ldx, C, es), {weight, (size_t)C * W * 4}, {bias, (size_t)C * 4}, {slots, (size_t)N * 4}};
    const Span out[] = {{y, (size_t)N * C * es}, {history, (size_t)P * (W - 1) * C * es}, {status, 4}};
    if (!apart(in, out)) return KDA_ERR_INVALID_ARG;
    cudaStream_t st = (cudaStream_t)stream;
    if (clear(status, st) != KDA_OK) return KDA_ERR_CUDA;
    if (N == 0) return KDA_OK;
    kda::ConvStepParams p{x, ldx, weight, bias, conv_act, history, slots, N, P, C, W, y, status};
    return from_cuda(kda::short_conv_step(dtype, p, st));
}

kda_status kda_ssm_step(const void* u, int64_t ldu, const void* delta, int64_t ldd, const float* A, const void* Bm,
                        int64_t ldb, const void* Cm, int64_t ldc, const float* D, const void* z, int64_t ldz,
                        const float* delta_bias, int softplus, kda_dtype dtype, float* state, const int32_t* slots,
                        int P, int N, int C, int G, int S, void* y, int32_t* status, void* stream) {
    if (N < 0 || P < 0 || C <= 0 || G <= 0 || C % G != 0) return KDA_ERR_INVALID_ARG;
    if (!dtype_ok(dtype) || (S != 8 && S != 16 && S != 32 && S != 64) || C > kMostChannels || N > kMostRows ||
        (slots && N > KDA_MOST_SLOTS))
        return KDA_ERR_UNSUPPORTED;
    if (softplus != 0 && softplus != 1) return KDA_ERR_INVALID_ARG;
    const int64_t vec = (int64_t)G * S;
    if (ldu < C || ldd < C || (z && ldz < C) || ldb < vec || ldc < vec) return KDA_ERR_INVALID_ARG;
    if (N > 0 && (!u || !delta || !A || !Bm || !Cm || !state || !y || P == 0)) return KDA_ERR_INVALID_ARG;
    if (!slots && N > P) return KDA_ERR_INVALID_ARG;
    if ((int64_t)N * (((int64_t)C * S + 1023) / 1024) > 0x7fffffffLL) return KDA_ERR_UNSUPPORTED;  // blocks of one launch
    const size_t es = size_of(dtype);
    for (const void* p : {u, delta, Bm, Cm, z, (const void*)y})
        if (!aligned(p, es)) return KDA_ERR_INVALID_ARG;
    if (!kda_host::aligned16(A) || !aligned(state, 32)) return KDA_ERR_INVALID_ARG;
    if (!aligned(D, 4) || !aligned(delta_bias, 4) || !aligned(slots, 4) || !aligned(status, 4)) return KDA_ERR_INVALID_ARG;
    const Span in[] = {rows(u, N, ldu, C, es), rows(delta, N, ldd, C, es), rows(z, N, ldz, C, es), rows(Bm, N, ldb, vec, es),
                       rows(Cm, N, ldc, vec, es), {A, (size_t)C * S * 4}, {D, (size_t)C * 4}, {delta_bias, (size_t)C * 4},
                       {slots, (size_t)N * 4}};
    const Span out[] = {{y, (size_t)N * C * es}, {state, (size_t)P * C * S * 4}, {status, 4}};
    if (!apart(in, out)) return KDA_ERR_INVALID_ARG;
    cudaStream_t st = (cudaStream_t)stream;
    if (clear(status, st) != KDA_OK) return KDA_ERR_CUDA;
    if (N == 0) return KDA_OK;
    kda::SsmStepParams p{};
    p.u = u; p.delta = delta; p.z = z; p.ldu = ldu; p.ldd = ldd; p.ldz = ldz;
    p.Bm = Bm; p.Cm = Cm; p.ldb = ldb; p.ldc = ldc;
    p.A = A; p.D = D; p.bias = delta_bias; p.softplus = softplus;
    p.state = state; p.slots = slots; p.N = N; p.P = P; p.C = C; p.G = G; p.S = S; p.y = y; p.status = status;
    return from_cuda(kda::ssm_step(dtype, p, st));
}

size_t kda_ssm_scan_fwd_workspace_size(int B, int T, int C, int G, int S, int N, int packed) {
    kda::SsmScanParams p{};
    if (scan_sizes(p, B, T, C, G, S, N, packed ? kPacked : nullptr) != KDA_OK) return 0;
    return kda::ssm_scan_workspace(p);
}

kda_status kda_ssm_scan_fwd(const void* u, int64_t ldu, const void* delta, int64_t ldd, const float* A, const void* Bm,
                            int64_t ldb, const void* Cm, int64_t ldc, const float* D, const void* z, int64_t ldz,
                            const float* delta_bias, int softplus, kda_dtype dtype, const float* initial_state,
                            const int32_t* cu_seqlens, int B, int T, int C, int G, int S, int N, void* y,
                            float* final_state, void* workspace, size_t workspace_bytes, void* stream) {
    kda::SsmScanParams p{};
    kda_status s = scan_sizes(p, B, T, C, G, S, N, cu_seqlens);
    if (s != KDA_OK) return s;
    p.u = u; p.delta = delta; p.z = z; p.ldu = ldu; p.ldd = ldd; p.ldz = ldz;
    p.Bm = Bm; p.Cm = Cm; p.ldb = ldb; p.ldc = ldc; p.A = A; p.D = D; p.bias = delta_bias; p.softplus = softplus;
    p.initial = initial_state; p.y = y; p.final_state = final_state; p.ws = workspace;
    if ((s = scan_inputs(p, dtype)) != KDA_OK) return s;
    const size_t es = size_of(dtype), need = kda::ssm_scan_workspace(p), states = (size_t)N * C * S * 4;
    if (p.total > 0 && !y) return KDA_ERR_INVALID_ARG;
    if (!aligned(y, es) || !kda_host::aligned16(final_state)) return KDA_ERR_INVALID_ARG;
    if (workspace_bytes < need || (need > 0 && !workspace)) return KDA_ERR_WORKSPACE;
    if (!kda_host::aligned16(workspace)) return KDA_ERR_INVALID_ARG;
    SCAN_INPUT_SPANS(in, p, es);
    const Span out[] = {{y, (size_t)p.total * C * es}, {final_state, states}, {workspace, need}};
    if (!apart(in, out)) return KDA_ERR_INVALID_ARG;
    if (N == 0) return KDA_OK;
    return from_cuda(kda::ssm_scan_fwd(dtype, p, (cudaStream_t)stream));
}

size_t kda_ssm_scan_bwd_workspace_size(int B, int T, int C, int G, int S, int N, int packed) {
    kda::SsmScanParams p{};
    if (scan_sizes(p, B, T, C, G, S, N, packed ? kPacked : nullptr) != KDA_OK) return 0;
    return kda::ssm_scan_bwd_workspace(p);
}

kda_status kda_ssm_scan_bwd(const void* u, int64_t ldu, const void* delta, int64_t ldd, const float* A, const void* Bm,
                            int64_t ldb, const void* Cm, int64_t ldc, const float* D, const void* z, int64_t ldz,
                            const float* delta_bias, int softplus, kda_dtype dtype, const float* initial_state,
                            const int32_t* cu_seqlens, int B, int T, int C, int G, int S, int N, const void* dy,
                            const float* dfinal_state, kda_dtype grad_dtype, void* du, void* ddelta, float* dA, void* dB,
                            void* dC, float* dD, void* dz, float* ddelta_bias, float* dinitial_state, void* workspace,
                            size_t workspace_bytes, void* stream) {
    kda::SsmScanParams p{};
    kda_status s = scan_sizes(p, B, T, C, G, S, N, cu_seqlens);
    if (s != KDA_OK) return s;
    if (p.total > kMostBwdTokens) return KDA_ERR_UNSUPPORTED;
    p.u = u; p.delta = delta; p.z = z; p.ldu = ldu; p.ldd = ldd; p.ldz = ldz;
    p.Bm = Bm; p.Cm = Cm; p.ldb = ldb; p.ldc = ldc; p.A = A; p.D = D; p.bias = delta_bias; p.softplus = softplus;
    p.initial = initial_state; p.ws = workspace;
    p.dy = dy; p.dfinal = dfinal_state; p.du = du; p.ddelta = ddelta; p.dz = dz; p.dB = dB; p.dC = dC;
    p.dA = dA; p.dD = dD; p.dbias = ddelta_bias; p.dinitial = dinitial_state;
    if (dtype_ok(dtype) && (!dtype_ok(grad_dtype) || (dtype == KDA_F32 && grad_dtype != KDA_F32))) return KDA_ERR_UNSUPPORTED;
    if ((s = scan_inputs(p, dtype)) != KDA_OK) return s;
    const size_t es = size_of(dtype), gs = size_of(grad_dtype), need = kda::ssm_scan_bwd_workspace(p);
    if (!dA || (p.total > 0 && (!dy || !du || !ddelta || !dB || !dC)) || (p.total > 0 && !z != !dz)) return KDA_ERR_INVALID_ARG;
    for (const void* q : {dy, (const void*)du, (const void*)ddelta, (const void*)dz, (const void*)dB, (const void*)dC})
        if (!aligned(q, gs)) return KDA_ERR_INVALID_ARG;
    for (const float* q : {dfinal_state, (const float*)dinitial_state})
        if (!kda_host::aligned16(q)) return KDA_ERR_INVALID_ARG;
    for (const float* q : {dA, dD, ddelta_bias})
        if (!aligned(q, 4)) return KDA_ERR_INVALID_ARG;
    if (workspace_bytes < need || !workspace) return KDA_ERR_WORKSPACE;
    if (!kda_host::aligned16(workspace)) return KDA_ERR_INVALID_ARG;
    const size_t rows_bytes = (size_t)p.total * C * gs, vec = (size_t)p.total * G * S * gs, states = (size_t)N * C * S * 4;
    SCAN_INPUT_SPANS(in, p, es);
    const Span more[] = {{dy, rows_bytes}, {dfinal_state, states}};
    const Span out[] = {{du, rows_bytes}, {ddelta, rows_bytes}, {dz, rows_bytes}, {dB, vec}, {dC, vec}, {dA, (size_t)C * S * 4},
                        {dD, (size_t)C * 4}, {ddelta_bias, (size_t)C * 4}, {dinitial_state, states}, {workspace, need}};
    if (!apart(in, out) || !apart(more, out)) return KDA_ERR_INVALID_ARG;
    return from_cuda(kda::ssm_scan_bwd(dtype, grad_dtype, p, (cudaStream_t)stream));
}

kda_status kda_pages_alloc(int32_t* refs, int P, int n, int32_t* pages, int32_t* status, void* stream) {
    if (n > kMostPages) return KDA_ERR_UNSUPPORTED;
    if (P < 0 || n < 0 || (P > 0 && !refs) || (n > 0 && !pages)) return KDA_ERR_INVALID_ARG;
    if (P > kMostPages) return KDA_ERR_UNSUPPORTED;
    if (!aligned(refs, 4) || !aligned(pages, 4) || !aligned(status, 4)) return KDA_ERR_INVALID_ARG;
    const Span in[] = {{nullptr, 0}};
    const Span out[] = {{refs, (size_t)P * 4}, {pages, (size_t)n * 4}, {status, 4}};
    if (!apart(in, out)) return KDA_ERR_INVALID_ARG;
    cudaStream_t st = (cudaStream_t)stream;
    if (clear(status, st) != KDA_OK) return KDA_ERR_CUDA;
    if (n == 0) return KDA_OK;
    return from_cuda(kda::pages_alloc(refs, P, n, pages, status, st));
}

kda_status kda_pages_free(int32_t* refs, int P, const int32_t* pages, int64_t n, int32_t* status, void* stream) {
    if (P < 0 || n < 0 || (P > 0 && !refs) || (n > 0 && !pages)) return KDA_ERR_INVALID_ARG;
    if (P > kMostPages) return KDA_ERR_UNSUPPORTED;
    if (!aligned(refs, 4) || !aligned(pages, 4) || !aligned(status, 4)) return KDA_ERR_INVALID_ARG;
    const Span in[] = {{pages, (size_t)n * 4}};
    const Span out[] = {{refs, (size_t)P * 4}, {status, 4}};
    if (!apart(in, out)) return KDA_ERR_INVALID_ARG;
    cudaStream_t st = (cudaStream_t)stream;
    if (clear(status, st) != KDA_OK) return KDA_ERR_CUDA;
    if (n == 0) return KDA_OK;
    return from_cuda(kda::pages_free(refs, P, pages, n, status, st));
}

kda_status kda_pages_fork(int32_t* tables, int32_t* lens, int S, int width, int page_tokens, int32_t* refs, int P,
                          const int32_t* parents, const int32_t* children, int n, int32_t* src, int32_t* dst,
                          int32_t* status, void* stream) {
    if (S < 0 || width <= 0 || page_tokens <= 0 || P < 0 || n < 0) return KDA_ERR_INVALID_ARG;
    if (n > 65536 || P > kMostPages) return KDA_ERR_UNSUPPORTED;
    if (n > 0 && (!parents || !children || !src || !dst)) return KDA_ERR_INVALID_ARG;
    if ((S > 0 && (!tables || !lens)) || (P > 0 && !refs)) return KDA_ERR_INVALID_ARG;
    for (const void* p : {(const void*)tables, (const void*)lens, (const void*)refs, (const void*)parents,
                          (const void*)children, (const void*)src, (const void*)dst, (const void*)status})
        if (!aligned(p, 4)) return KDA_ERR_INVALID_ARG;
    const size_t list = (size_t)n * 4;
    const Span in[] = {{parents, list}, {children, list}};
    const Span out[] = {{tables, (size_t)S * width * 4}, {lens, (size_t)S * 4}, {refs, (size_t)P * 4}, {src, list}, {dst, list},
                        {status, 4}};
    if (!apart(in, out)) return KDA_ERR_INVALID_ARG;
    cudaStream_t st = (cudaStream_t)stream;
    if (clear(status, st) != KDA_OK) return KDA_ERR_CUDA;
    if (n == 0) return KDA_OK;
    return from_cuda(kda::pages_fork(tables, lens, S, width, page_tokens, refs, P, parents, children, n, src, dst, status, st));
}

size_t kda_pages_compact_workspace_size(int P) { return P <= 0 ? 0 : kda::pages_compact_workspace(P); }

kda_status kda_pages_compact(int32_t* refs, int P, int32_t* tables, int64_t entries, int32_t* src, int32_t* dst,
                             void* workspace, size_t workspace_bytes, int32_t* status, void* stream) {
    if (P < 0 || entries < 0 || (P > 0 && !refs) || (entries > 0 && !tables) || (P > 1 && (!src || !dst))) return KDA_ERR_INVALID_ARG;
    if (P > kMostPages) return KDA_ERR_UNSUPPORTED;
    for (const void* p : {(const void*)tables, (const void*)refs, (const void*)src, (const void*)dst, (const void*)status})
        if (!aligned(p, 4)) return KDA_ERR_INVALID_ARG;
    const size_t need = P > 0 ? kda::pages_compact_workspace(P) : 0;
    if (workspace_bytes < need || (need > 0 && !workspace)) return KDA_ERR_WORKSPACE;
    if (!kda_host::aligned16(workspace)) return KDA_ERR_INVALID_ARG;
    const Span in[] = {{nullptr, 0}};
    const Span out[] = {{tables, (size_t)entries * 4}, {refs, (size_t)P * 4}, {src, (size_t)(P / 2) * 4},
                        {dst, (size_t)(P / 2) * 4}, {workspace, need}, {status, 4}};
    if (!apart(in, out)) return KDA_ERR_INVALID_ARG;
    cudaStream_t st = (cudaStream_t)stream;
    if (clear(status, st) != KDA_OK) return KDA_ERR_CUDA;
    if (P == 0) return KDA_OK;
    return from_cuda(kda::pages_compact(refs, P, tables, entries, src, dst, workspace, status, st));
}

size_t kda_pages_copy_workspace_size(int P, int n) { return P <= 0 || n <= 0 ? 0 : kda::pages_copy_workspace(P, n); }

kda_status kda_pages_copy(void* pool, int P, int64_t page_bytes, const int32_t* src, const int32_t* dst, int n,
                          void* workspace, size_t workspace_bytes, int32_t* status, void* stream) {
    if (P < 0 || n < 0 || page_bytes <= 0 || (P > 0 && !pool) || (n > 0 && (!src || !dst))) return KDA_ERR_INVALID_ARG;
    if (page_bytes % 16 != 0 || P > kMostPages || n > kMostPages) return KDA_ERR_UNSUPPORTED;
    if ((double)P * (double)page_bytes > 9.0e18) return KDA_ERR_INVALID_ARG;
    if (!kda_host::aligned16(pool) || !aligned(src, 4) || !aligned(dst, 4) || !aligned(status, 4)) return KDA_ERR_INVALID_ARG;
    const size_t need = P > 0 && n > 0 ? kda::pages_copy_workspace(P, n) : 0;
    if (workspace_bytes < need || (need > 0 && !workspace)) return KDA_ERR_WORKSPACE;
    if (!kda_host::aligned16(workspace)) return KDA_ERR_INVALID_ARG;
    const Span in[] = {{src, (size_t)n * 4}, {dst, (size_t)n * 4}};
    const Span out[] = {{pool, (size_t)P * page_bytes}, {workspace, need}, {status, 4}};
    if (!apart(in, out)) return KDA_ERR_INVALID_ARG;
    cudaStream_t st = (cudaStream_t)stream;
    if (clear(status, st) != KDA_OK) return KDA_ERR_CUDA;
    if (P == 0 || n == 0) return KDA_OK;
    return from_cuda(kda::pages_copy(pool, P, page_bytes, src, dst, n, workspace, status, st));
}

}  // extern "C"
