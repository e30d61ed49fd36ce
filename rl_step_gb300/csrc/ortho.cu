// mlora_orthogonalize (include/mlora.h): checks, and the kernel's table of matrices
// (ortho_kernel.cuh).
#include <cfloat>
#include <new>
#include <vector>

#include "kv_common.cuh"
#include "ortho.cuh"

using namespace mlk;

extern "C" int mlora_orthogonalize(const mlora_matrix_set* m, const mlora_newton_schulz* p, void* stream) try {
    if (!m || !p) return kv_fail(MLORA_E_ARG, "NULL matrices or parameters");
    if (m->n_matrices < 0) return kv_fail(MLORA_E_ARG, "%d matrices", m->n_matrices);
    if (m->dtype != MLORA_BF16 && m->dtype != MLORA_FP32) return kv_fail(MLORA_E_ARG, "unknown dtype %d", m->dtype);
    if (m->n_matrices > 0 && (!m->src || !m->rows || !m->cols)) return kv_fail(MLORA_E_ARG, "NULL matrix or size array");
    if (p->steps < 1 || p->steps > MLORA_ORTHO_MAX_STEPS)
        return kv_fail(MLORA_E_ARG, "%d steps, 1 .. %d are possible", p->steps, MLORA_ORTHO_MAX_STEPS);
    if (!(fabsf(p->a) <= FLT_MAX && fabsf(p->b) <= FLT_MAX && fabsf(p->c) <= FLT_MAX) || !(p->eps > 0.f && p->eps <= FLT_MAX))
        return kv_fail(MLORA_E_ARG, "coefficients must be finite, eps positive");
    const uintptr_t es = m->dtype == MLORA_BF16 ? 2 : 4;
    std::vector<OrthoEntry> e;
    e.reserve(m->n_matrices);
    for (int i = 0; i < m->n_matrices; ++i) {
        const int64_t rows = m->rows[i], cols = m->cols[i];
        if (rows < 0 || cols < 0 || rows > INT32_MAX - 4096 || cols > INT32_MAX - 4096)
            return kv_fail(MLORA_E_ARG, "matrix %d: %lld x %lld", i, (long long)rows, (long long)cols);
        if (rows == 0 || cols == 0) continue;
        const int64_t r = rows < cols ? rows : cols;
        if (r > MLORA_MAX_RANK)
            return kv_fail(MLORA_E_ARG, "matrix %d: %lld x %lld, the shorter side is at most %d", i, (long long)rows,
                           (long long)cols, MLORA_MAX_RANK);
        const void* src = m->src[i];
        void* dst = m->dst ? m->dst[i] : const_cast<void*>(src);
        if (!src || !dst) return kv_fail(MLORA_E_ARG, "matrix %d is NULL", i);
        const uintptr_t both = reinterpret_cast<uintptr_t>(src) | reinterpret_cast<uintptr_t>(dst);
        if (both % es) return kv_fail(MLORA_E_ARG, "matrix %d is not aligned to its elements", i);
        OrthoEntry x;
        x.src = src;
        x.dst = dst;
        x.n = (int)(rows < cols ? cols : rows);
        x.r = (int16_t)r;
        x.tall = rows > cols;
        x.vec = both % (4 * es) == 0 && cols % 4 == 0;
        e.push_back(x);
    }
    const OrthoCoeffs co{p->a, p->b, p->c, p->eps, p->steps};
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (e.empty()) return MLORA_OK;
    int dev = 0, sms = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err == cudaSuccess) err = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (err == cudaSuccess) err = m->dtype == MLORA_BF16 ? launch_ortho_bf16(e, co, sms, s) : launch_ortho_fp32(e, co, sms, s);
    if (err != cudaSuccess) return kv_fail(MLORA_E_CUDA, "orthogonalising: %s", cudaGetErrorString(err));
    return MLORA_OK;
} catch (const std::bad_alloc&) {
    return kv_fail(MLORA_E_NOMEM, "no host memory for the matrix table");
}
