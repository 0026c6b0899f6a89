// api_grads.hip -- the C-ABI entry points of the gradients' norm and clipping.
// Argument checks as in api.hip: every error is a status, before anything is
// enqueued.
#include "gemm_f32.h"
#include "api_checks.h"
#include "grad_norm.h"

#include <algorithm>
#include <math.h>
#include <stdlib.h>

namespace gemmf32 {
namespace {

int check_sizes(int64_t count, const int64_t* sizes) {
    if (count < 0) return GEMM_F32_ERR_INVALID_DIM;
    if (count > INT_MAX) return GEMM_F32_ERR_TOO_LARGE;
    if (count > 0 && sizes == nullptr) return GEMM_F32_ERR_NULL_PTR;
    for (int64_t i = 0; i < count; ++i) {
        if (sizes[i] < 0) return GEMM_F32_ERR_INVALID_DIM;
        if (sizes[i] > (int64_t)1 << 42) return GEMM_F32_ERR_TOO_LARGE;
    }
    return GEMM_F32_OK;
}

int check_tensors(int64_t count, const void* const* data, const int64_t* sizes, const int* types) {
    const int st = check_sizes(count, sizes);
    if (st != GEMM_F32_OK) return st;
    if (count > 0 && (data == nullptr || types == nullptr)) return GEMM_F32_ERR_NULL_PTR;
    for (int64_t i = 0; i < count; ++i) {
        if (!known_type(types[i])) return GEMM_F32_ERR_INVALID_TYPE;
        if (sizes[i] > 0 && data[i] == nullptr) return GEMM_F32_ERR_NULL_PTR;
        if (misaligned_type(data[i], types[i])) return GEMM_F32_ERR_MISALIGNED;
    }
    return GEMM_F32_OK;
}

// Blocks write outputs while others still read: an output may be its own
// input, and overlap nothing else.  The norm is one more input, or, where it is
// written (by a block of the same launch), one more output.
struct Range {
    uintptr_t begin, end;
    bool output;
};
int check_overlaps(const GradList& l, const float* norm, bool written) {
    Range few[513];
    Range* r = few;
    if (l.count > 256) {
        r = static_cast<Range*>(malloc((2 * (size_t)l.count + 1) * sizeof(Range)));
        if (r == nullptr) return GEMM_F32_ERR_TOO_LARGE;
    }
    int64_t n = 0;
    r[n++] = Range{(uintptr_t)norm, (uintptr_t)norm + sizeof(float), written};
    for (int64_t i = 0; i < l.count; ++i) {
        if (l.size[i] == 0) continue;
        const uintptr_t in = (uintptr_t)l.in[i], out = (uintptr_t)l.out[i];
        const uintptr_t bytes = (uintptr_t)l.size[i] * (l.type[i] == GEMM_MIXED_F32 ? 4 : 2);
        r[n++] = Range{out, out + bytes, true};
        if (in != out) r[n++] = Range{in, in + bytes, false};
    }
    std::sort(r, r + n, [](const Range& a, const Range& b) { return a.begin < b.begin; });
    uintptr_t outputs = 0, any = 0;                // ends so far
    int st = GEMM_F32_OK;
    for (int64_t i = 0; i < n; ++i) {
        if (r[i].begin < (r[i].output ? any : outputs)) st = GEMM_F32_ERR_OVERLAP;
        any = std::max(any, r[i].end);
        if (r[i].output) outputs = std::max(outputs, r[i].end);
    }
    if (r != few) free(r);
    return st;
}

int check_clip(const GradList& l, float max_norm, float eps, const float* norm, bool written) {
    int st = check_tensors(l.count, l.in, l.size, l.type);
    if (st != GEMM_F32_OK) return st;
    if (!(max_norm >= 0.0f) || !isfinite(max_norm) || !(eps > 0.0f) || !isfinite(eps)) return GEMM_F32_ERR_INVALID_SCALAR;
    if (norm == nullptr || (l.count > 0 && l.out == nullptr)) return GEMM_F32_ERR_NULL_PTR;
    if (misaligned(norm)) return GEMM_F32_ERR_MISALIGNED;
    for (int64_t i = 0; i < l.count; ++i) {
        if (l.size[i] > 0 && l.out[i] == nullptr) return GEMM_F32_ERR_NULL_PTR;
        if (misaligned_type(l.out[i], l.type[i])) return GEMM_F32_ERR_MISALIGNED;
    }
    return check_overlaps(l, norm, written);
}

}  // namespace
}  // namespace gemmf32

using namespace gemmf32;

extern "C" int64_t grad_norm_workspace_size(int64_t count, const int64_t* sizes) {
    if (check_sizes(count, sizes) != GEMM_F32_OK) return -1;
    return 8 * grad_partials(count, sizes);
}

extern "C" int grad_norm(int64_t count, const void* const* grads, const int64_t* sizes, const int* types, float* norm,
                         void* workspace, int64_t workspace_bytes, void* stream) {
    int st = check_tensors(count, grads, sizes, types);
    if (st != GEMM_F32_OK) return st;
    if (norm == nullptr) return GEMM_F32_ERR_NULL_PTR;
    if (misaligned(norm)) return GEMM_F32_ERR_MISALIGNED;
    const int64_t partials = grad_partials(count, sizes);
    st = check_workspace(8 * partials, workspace, workspace_bytes);
    if (st != GEMM_F32_OK) return st;
    if ((st = check_device()) != GEMM_F32_OK) return st;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    const GradList l{count, grads, nullptr, sizes, types};
    hipError_t e = launch_grad_squares(l, static_cast<double*>(workspace), s);
    if (e == hipSuccess) e = launch_grad_norm(static_cast<double*>(workspace), partials, norm, s);
    return finish(e);
}

extern "C" int grad_clip(int64_t count, const void* const* grads, void* const* out, const int64_t* sizes,
                         const int* types, const float* norm, float max_norm, float eps, void* stream) {
    const GradList l{count, grads, out, sizes, types};
    int st = check_clip(l, max_norm, eps, norm, false);
    if (st != GEMM_F32_OK) return st;
    if ((st = check_device()) != GEMM_F32_OK) return st;
    return finish(launch_grad_clip(l, nullptr, 0, const_cast<float*>(norm), max_norm, eps,
                                   reinterpret_cast<hipStream_t>(stream)));
}

extern "C" int grad_clip_norm(int64_t count, const void* const* grads, void* const* out, const int64_t* sizes,
                              const int* types, float max_norm, float eps, float* norm, void* workspace,
                              int64_t workspace_bytes, void* stream) {
    const GradList l{count, grads, out, sizes, types};
    int st = check_clip(l, max_norm, eps, norm, true);
    if (st != GEMM_F32_OK) return st;
    const int64_t partials = grad_partials(count, sizes);
    st = check_workspace(8 * partials, workspace, workspace_bytes);
    if (st != GEMM_F32_OK) return st;
    if ((st = check_device()) != GEMM_F32_OK) return st;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    double* const sums = static_cast<double*>(workspace);
    if (partials == 0) return finish(launch_grad_norm(sums, 0, norm, s));
    hipError_t e = launch_grad_squares(l, sums, s);
    if (e == hipSuccess) e = launch_grad_clip(l, sums, partials, norm, max_norm, eps, s);
    return finish(e);
}
