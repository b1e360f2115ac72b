// qmm_api.hip -- the exported C ABI: argument checks in the documented
// order, then dispatch to the launchers.  Nothing here allocates.
#include <math.h>
#include <stdarg.h>
#include <string.h>

#include <cstdio>
#include <string>

#include "../../include/qmm.h"
#include "qmm_internal.h"

#define QMM_EXPORT extern "C" __attribute__((visibility("default")))

namespace {

thread_local std::string g_last_error;

int fail(int status, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
int fail(int status, const char *fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  g_last_error = buf;
  return status;
}

int ok() {
  g_last_error.clear();
  return QMM_OK;
}

struct KindInfo {
  int id;
  const char *name;
  int block_bytes;
  int block_elems;
};

// The kind table (GGUF type ids; ferrox-cuda 0.21.0 mul_mm.rs, KINDS).
constexpr KindInfo kKinds[] = {
    {QMM_Q8_0, "Q8_0", 34, 32},     {QMM_Q4_0, "Q4_0", 18, 32},     {QMM_Q5_0, "Q5_0", 22, 32},
    {QMM_Q2_K, "Q2_K", 84, 256},    {QMM_Q3_K, "Q3_K", 110, 256},   {QMM_Q4_K, "Q4_K", 144, 256},
    {QMM_Q5_K, "Q5_K", 176, 256},   {QMM_Q6_K, "Q6_K", 210, 256},   {QMM_IQ4_NL, "IQ4_NL", 18, 32},
    {QMM_IQ4_XS, "IQ4_XS", 136, 256}, {QMM_MXFP4, "MXFP4", 17, 32},
};

const KindInfo *find_kind(int kind) {
  for (const KindInfo &k : kKinds)
    if (k.id == kind) return &k;
  return nullptr;
}

bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

// Empty shape, then kind, then K alignment: the order of ferrox-cuda
// mul_mm.rs validate_shape.  K and the per-launch sizes must also fit the
// kernels' 32-bit indices.
int check_shape(int kind, int64_t M, int64_t N, int64_t K, const KindInfo **out) {
  if (M <= 0 || N <= 0 || K <= 0)
    return fail(QMM_ERR_EMPTY_SHAPE, "empty shape: M=%lld N=%lld K=%lld", (long long)M, (long long)N,
                (long long)K);
  const KindInfo *k = find_kind(kind);
  if (!k) return fail(QMM_ERR_UNSUPPORTED_KIND, "kind %d is not one of the eleven supported kinds", kind);
  if (K % k->block_elems != 0)
    return fail(QMM_ERR_K_NOT_BLOCK_ALIGNED, "K=%lld is not a whole number of %s blocks (%d elements)",
                (long long)K, k->name, k->block_elems);
  if (K > (int64_t)1 << 30 || N > (int64_t)INT32_MAX)
    return fail(QMM_ERR_BAD_ARG, "K=%lld or N=%lld exceeds the supported range", (long long)K,
                (long long)N);
  *out = k;
  return QMM_OK;
}

int check_dtype(int dtype) {
  if (dtype != QMM_F32 && dtype != QMM_F16) return fail(QMM_ERR_BAD_DTYPE, "dtype %d is neither QMM_F32 nor QMM_F16", dtype);
  return QMM_OK;
}

int check_act(const void *x, int dtype, const char *what) {
  if (!x) return fail(QMM_ERR_BAD_ARG, "%s is NULL", what);
  if (!aligned(x, dtype == QMM_F32 ? 4 : 2))
    return fail(QMM_ERR_BAD_ARG, "%s is not aligned to its element size", what);
  return QMM_OK;
}

int hip_status(hipError_t e, const char *what) {
  if (e != hipSuccess) return fail(QMM_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
  return ok();
}

}  // namespace

QMM_EXPORT int qmm_gemv_ex(int kind, const void *W, const void *x, int x_dtype, float *y, int64_t M,
                           int64_t N, int64_t K, void *stream) {
  const KindInfo *k;
  int st = check_shape(kind, M, N, K, &k);
  if (st) return st;
  if ((st = check_dtype(x_dtype))) return st;
  if (!W || !y) return fail(QMM_ERR_BAD_ARG, "W or y is NULL");
  if ((st = check_act(x, x_dtype, "x"))) return st;
  if (!aligned(y, 4)) return fail(QMM_ERR_BAD_ARG, "y is not 4-byte aligned");
  if (M > QMM_GEMV_MAX_M) return fail(QMM_ERR_BAD_ARG, "GEMV takes 1..%d tokens, got M=%lld", QMM_GEMV_MAX_M, (long long)M);
  return hip_status(qmm::launch_gemv(kind, (const uint8_t *)W, x, x_dtype == QMM_F16, y, (int)M, N, K,
                                     (hipStream_t)stream),
                    "gemv launch");
}

QMM_EXPORT int qmm_gemv(int kind, const void *W, const float *x, float *y, int64_t N, int64_t K) {
  return qmm_gemv_ex(kind, W, x, QMM_F32, y, 1, N, K, nullptr);
}

QMM_EXPORT int qmm_gemm_ex(int kind, const void *W, const void *A, int a_dtype, float *C, int64_t M,
                           int64_t N, int64_t K, void *stream) {
  const KindInfo *k;
  int st = check_shape(kind, M, N, K, &k);
  if (st) return st;
  if ((st = check_dtype(a_dtype))) return st;
  if (!W || !C) return fail(QMM_ERR_BAD_ARG, "W or C is NULL");
  if ((st = check_act(A, a_dtype, "A"))) return st;
  if (!aligned(C, 4)) return fail(QMM_ERR_BAD_ARG, "C is not 4-byte aligned");
  if (M > (int64_t)65535 * 64) return fail(QMM_ERR_BAD_ARG, "M=%lld exceeds the supported range", (long long)M);
  return hip_status(qmm::launch_gemm(kind, (const uint8_t *)W, A, a_dtype == QMM_F16, C, M, N, K,
                                     (hipStream_t)stream),
                    "gemm launch");
}

QMM_EXPORT int qmm_gemm(int kind, const void *W, const void *A, float *C, int64_t M, int64_t N, int64_t K) {
  return qmm_gemm_ex(kind, W, A, QMM_F16, C, M, N, K, nullptr);
}

QMM_EXPORT int qmm_matmul(int kind, const void *W, const void *A, int a_dtype, float *C, int64_t M,
                          int64_t N, int64_t K, void *stream) {
  if (M >= 1 && M <= QMM_GEMV_MAX_M) return qmm_gemv_ex(kind, W, A, a_dtype, C, M, N, K, stream);
  return qmm_gemm_ex(kind, W, A, a_dtype, C, M, N, K, stream);
}

QMM_EXPORT size_t qmm_moe_ffn_workspace_bytes(int64_t E, int64_t M, int64_t topk, int64_t N_ff, int64_t K) {
  if (E <= 0 || M <= 0 || topk <= 0 || N_ff <= 0 || K <= 0) return 0;
  return qmm::moe_ffn_workspace_bytes(E, M, topk, N_ff, K);
}

// Kind, then K % 256 (the repacked layout's k-block), after the usual shape
// checks.
static int check_packed(int kind, int64_t M, int64_t N, int64_t K) {
  const KindInfo *k;
  int st = check_shape(kind, M, N, K, &k);
  if (st) return st;
  if (!qmm::packed_supported(kind))
    return fail(QMM_ERR_UNSUPPORTED_KIND, "%s has no repacked layout", k->name);
  if (K % 256 != 0)
    return fail(QMM_ERR_K_NOT_BLOCK_ALIGNED, "the repacked layout needs K a multiple of 256, got K=%lld",
                (long long)K);
  if (qmm::packed_bytes_of(kind, N, K) > ((int64_t)1 << 40))
    return fail(QMM_ERR_BAD_ARG, "N=%lld, K=%lld exceed the supported range", (long long)N, (long long)K);
  return QMM_OK;
}

static int moe_ffn_checked(int kind, const void *W_gu, const void *W_d, int64_t E, const int32_t *ids,
                           const float *topk_w, int64_t topk, const void *X, int x_dtype, float *Y, int64_t M,
                           int64_t N_ff, int64_t K, void *workspace, size_t workspace_bytes, void *stream,
                           bool packed) {
  const KindInfo *k;
  if (E <= 0 || topk <= 0 || N_ff <= 0)
    return fail(QMM_ERR_EMPTY_SHAPE, "empty shape: E=%lld topk=%lld N_ff=%lld", (long long)E, (long long)topk,
                (long long)N_ff);
  int st = check_shape(kind, M, 2 * N_ff, K, &k);  // gate/up: 2 N_ff rows of K
  if (st) return st;
  if ((st = check_shape(kind, M, K, N_ff, &k))) return st;  // down: K rows of N_ff
  if (packed) {
    if ((st = check_packed(kind, M, 2 * N_ff, K))) return st;
    if ((st = check_packed(kind, M, K, N_ff))) return st;
  }
  if ((st = check_dtype(x_dtype))) return st;
  if (!W_gu || !W_d || !ids || !topk_w || !Y) return fail(QMM_ERR_BAD_ARG, "W_gu, W_d, ids, topk_w or Y is NULL");
  if (packed && (!aligned(W_gu, 16) || !aligned(W_d, 16)))
    return fail(QMM_ERR_BAD_ARG, "the repacked W_gu or W_d is not 16-byte aligned");
  if ((st = check_act(X, x_dtype, "X"))) return st;
  if (!aligned(ids, 4) || !aligned(topk_w, 4)) return fail(QMM_ERR_BAD_ARG, "ids or topk_w is not 4-byte aligned");
  if (!aligned(Y, 16)) return fail(QMM_ERR_BAD_ARG, "Y is not 16-byte aligned");
  if (E > qmm::kMoeMaxExperts) return fail(QMM_ERR_BAD_ARG, "E=%lld exceeds %lld experts", (long long)E, (long long)qmm::kMoeMaxExperts);
  const int64_t P = M * topk;
  if (P > ((int64_t)1 << 31) - 1 || P * (N_ff > K ? 2 * N_ff : K) > ((int64_t)1 << 38) ||
      2 * N_ff > ((int64_t)1 << 31) / 4 || K > ((int64_t)1 << 31) / 4)
    return fail(QMM_ERR_BAD_ARG, "M*topk=%lld with N_ff=%lld, K=%lld exceeds the supported range", (long long)P,
                (long long)N_ff, (long long)K);
  // Repacked experts always run on the matrix cores, whose activation
  // offsets are 32-bit.
  if (packed && P * (N_ff > K ? N_ff : K) >= ((int64_t)1 << 31))
    return fail(QMM_ERR_BAD_ARG, "M*topk*max(K, N_ff)=%lld exceeds 2^31-1", (long long)(P * (N_ff > K ? N_ff : K)));
  const size_t need = qmm::moe_ffn_workspace_bytes(E, M, topk, N_ff, K);
  if (!workspace || workspace_bytes < need || !aligned(workspace, 256))
    return fail(QMM_ERR_WORKSPACE, "workspace needs %zu bytes (256-byte aligned), got %zu", need,
                workspace ? workspace_bytes : (size_t)0);
  return hip_status(qmm::launch_moe_ffn(kind, (const uint8_t *)W_gu, (const uint8_t *)W_d, E, ids, topk_w, topk, X,
                                        x_dtype == QMM_F16, Y, M, N_ff, K, workspace, (hipStream_t)stream, packed),
                    "moe_ffn launch");
}

QMM_EXPORT int qmm_moe_ffn(int kind, const void *W_gu, const void *W_d, int64_t E, const int32_t *ids,
                           const float *topk_w, int64_t topk, const void *X, int x_dtype, float *Y, int64_t M,
                           int64_t N_ff, int64_t K, void *workspace, size_t workspace_bytes, void *stream) {
  return moe_ffn_checked(kind, W_gu, W_d, E, ids, topk_w, topk, X, x_dtype, Y, M, N_ff, K, workspace,
                         workspace_bytes, stream, false);
}

QMM_EXPORT int qmm_moe_ffn_packed(int kind, const void *P_gu, const void *P_d, int64_t E, const int32_t *ids,
                                  const float *topk_w, int64_t topk, const void *X, int x_dtype, float *Y, int64_t M,
                                  int64_t N_ff, int64_t K, void *workspace, size_t workspace_bytes, void *stream) {
  return moe_ffn_checked(kind, P_gu, P_d, E, ids, topk_w, topk, X, x_dtype, Y, M, N_ff, K, workspace,
                         workspace_bytes, stream, true);
}

QMM_EXPORT size_t qmm_gemm_mx_workspace_bytes(int64_t M, int64_t K) {
  if (M <= 0 || K <= 0 || K % 32 != 0) return 0;
  return qmm::gemm_mx_workspace_bytes(M, K);
}

QMM_EXPORT int qmm_gemm_mx(int kind, const void *W, const void *A, int a_dtype, float *C, int64_t M, int64_t N,
                           int64_t K, void *workspace, size_t workspace_bytes, void *stream) {
  const KindInfo *k;
  int st = check_shape(kind, M, N, K, &k);
  if (st) return st;
  if (kind != QMM_MXFP4)
    return fail(QMM_ERR_UNSUPPORTED_KIND, "the scaled FP4 GEMM takes MXFP4 weights only, not kind %d", kind);
  if ((st = check_dtype(a_dtype))) return st;
  if (!W || !C) return fail(QMM_ERR_BAD_ARG, "W or C is NULL");
  if (!aligned(W, 16)) return fail(QMM_ERR_BAD_ARG, "W is not 16-byte aligned");
  if ((st = check_act(A, a_dtype, "A"))) return st;
  if (!aligned(C, 4)) return fail(QMM_ERR_BAD_ARG, "C is not 4-byte aligned");
  // One workgroup per 64 x 128 or 64 x 192 tile in a one-dimensional grid.
  const int64_t Mp = (M + 63) / 64 * 64;
  if (M > (int64_t)65535 * 64 || (Mp / 64) * ((N + 127) / 128) > (int64_t)INT32_MAX - 7 ||
      Mp * K > ((int64_t)1 << 40))
    return fail(QMM_ERR_BAD_ARG, "M=%lld, N=%lld, K=%lld exceed the supported range", (long long)M,
                (long long)N, (long long)K);
  const size_t need = qmm::gemm_mx_workspace_bytes(M, K);
  if (!workspace || workspace_bytes < need || !aligned(workspace, 16))
    return fail(QMM_ERR_WORKSPACE, "workspace needs %zu bytes at 16-byte alignment, got %zu", need,
                workspace ? workspace_bytes : (size_t)0);
  return hip_status(qmm::launch_gemm_mx((const uint8_t *)W, A, a_dtype == QMM_F16, C, M, N, K, workspace,
                                        (hipStream_t)stream),
                    "gemm_mx launch");
}

QMM_EXPORT size_t qmm_moe_workspace_bytes(int64_t E, int64_t M, int64_t topk) {
  if (E <= 0 || M < 0 || topk <= 0) return 0;
  return qmm::moe_workspace_bytes(E, M, topk);
}

QMM_EXPORT int qmm_moe(int kind, const void *W, int64_t E, const int32_t *ids, int64_t topk, const void *X,
                       int x_dtype, int x_per_slot, float *Y, int64_t M, int64_t N, int64_t K, void *workspace,
                       size_t workspace_bytes, void *stream) {
  const KindInfo *k;
  if (E <= 0 || topk <= 0)
    return fail(QMM_ERR_EMPTY_SHAPE, "empty shape: E=%lld topk=%lld", (long long)E, (long long)topk);
  int st = check_shape(kind, M, N, K, &k);
  if (st) return st;
  if ((st = check_dtype(x_dtype))) return st;
  if (!W || !ids || !Y) return fail(QMM_ERR_BAD_ARG, "W, ids or Y is NULL");
  if ((st = check_act(X, x_dtype, "X"))) return st;
  if (!aligned(ids, 4) || !aligned(Y, 4)) return fail(QMM_ERR_BAD_ARG, "ids or Y is not 4-byte aligned");
  if (x_per_slot != 0 && x_per_slot != 1) return fail(QMM_ERR_BAD_ARG, "x_per_slot must be 0 or 1");
  if (E > qmm::kMoeMaxExperts) return fail(QMM_ERR_BAD_ARG, "E=%lld exceeds %lld experts", (long long)E, (long long)qmm::kMoeMaxExperts);
  if (M * topk > ((int64_t)1 << 31) - 1) return fail(QMM_ERR_BAD_ARG, "M*topk exceeds 2^31-1");
  if (N > ((int64_t)1 << 31) / 4) return fail(QMM_ERR_BAD_ARG, "N=%lld exceeds the supported range", (long long)N);
  const size_t need = qmm::moe_workspace_bytes(E, M, topk);
  if (!workspace || workspace_bytes < need || !aligned(workspace, 4))
    return fail(QMM_ERR_WORKSPACE, "workspace needs %zu bytes (4-byte aligned), got %zu", need, workspace_bytes);
  return hip_status(qmm::launch_moe(kind, (const uint8_t *)W, E, ids, topk, X, x_dtype == QMM_F16, x_per_slot,
                                    Y, M, N, K, workspace, (hipStream_t)stream),
                    "moe launch");
}

QMM_EXPORT int64_t qmm_packed_bytes(int kind, int64_t N, int64_t K) {
  if (!qmm::packed_supported(kind)) return -1;
  return qmm::packed_bytes_of(kind, N, K);
}

QMM_EXPORT int qmm_repack(int kind, const void *W, void *P, int64_t N, int64_t K, void *stream) {
  int st = check_packed(kind, 1, N, K);
  if (st) return st;
  if (!W || !P) return fail(QMM_ERR_BAD_ARG, "W or P is NULL");
  if (!aligned(P, 16)) return fail(QMM_ERR_BAD_ARG, "P is not 16-byte aligned");
  return hip_status(qmm::launch_repack(kind, (const uint8_t *)W, P, N, K, (hipStream_t)stream), "repack launch");
}

QMM_EXPORT int qmm_gemv_packed(int kind, const void *P, const void *x, int x_dtype, float *y, int64_t M, int64_t N,
                               int64_t K, void *stream) {
  int st = check_packed(kind, M, N, K);
  if (st) return st;
  if ((st = check_dtype(x_dtype))) return st;
  if (!P || !y) return fail(QMM_ERR_BAD_ARG, "P or y is NULL");
  if (!aligned(P, 16)) return fail(QMM_ERR_BAD_ARG, "P is not 16-byte aligned");
  if ((st = check_act(x, x_dtype, "x"))) return st;
  if (!aligned(y, 4)) return fail(QMM_ERR_BAD_ARG, "y is not 4-byte aligned");
  if (M > QMM_GEMV_MAX_M) return fail(QMM_ERR_BAD_ARG, "GEMV takes 1..%d tokens, got M=%lld", QMM_GEMV_MAX_M, (long long)M);
  if (M * K >= ((int64_t)1 << 31)) return fail(QMM_ERR_BAD_ARG, "M*K=%lld exceeds 2^31-1", (long long)(M * K));
  return hip_status(qmm::launch_gemv_packed(kind, (const uint8_t *)P, x, x_dtype == QMM_F16, y, (int)M, N, K,
                                            (hipStream_t)stream),
                    "gemv_packed launch");
}

QMM_EXPORT int qmm_matmul_packed(int kind, const void *P, const void *A, int a_dtype, float *C, int64_t M, int64_t N,
                                 int64_t K, void *stream) {
  int st = check_packed(kind, M, N, K);
  if (st) return st;
  if ((st = check_dtype(a_dtype))) return st;
  if (!P || !C) return fail(QMM_ERR_BAD_ARG, "P or C is NULL");
  if (!aligned(P, 16)) return fail(QMM_ERR_BAD_ARG, "P is not 16-byte aligned");
  if ((st = check_act(A, a_dtype, "A"))) return st;
  if (!aligned(C, 4)) return fail(QMM_ERR_BAD_ARG, "C is not 4-byte aligned");
  if (M * K >= ((int64_t)1 << 31)) return fail(QMM_ERR_BAD_ARG, "M*K=%lld exceeds 2^31-1", (long long)(M * K));
  if (M <= QMM_GEMV_MAX_M)
    return hip_status(qmm::launch_gemv_packed(kind, (const uint8_t *)P, A, a_dtype == QMM_F16, C, (int)M, N, K,
                                              (hipStream_t)stream),
                      "matmul_packed launch (GEMV)");
  if (!qmm::gemm_packed_supported(kind))
    return fail(QMM_ERR_UNSUPPORTED_KIND, "the prefill GEMM over repacked weights does not take kind %d (M > %d)",
                kind, QMM_GEMV_MAX_M);
  // The GEMM addresses P and A through buffer descriptors with signed 32-bit
  // byte offsets.
  const int64_t a_bytes = M * K * (a_dtype == QMM_F16 ? 2 : 4);
  if (qmm::packed_bytes_of(kind, N, K) >= ((int64_t)1 << 31) || a_bytes >= ((int64_t)1 << 31) ||
      M >= ((int64_t)1 << 24))
    return fail(QMM_ERR_BAD_ARG, "N=%lld, K=%lld, M=%lld exceed the GEMM's 32-bit offsets", (long long)N,
                (long long)K, (long long)M);
  return hip_status(qmm::launch_gemm_packed(kind, (const uint8_t *)P, A, a_dtype == QMM_F16, C, M, N, K,
                                            (hipStream_t)stream),
                    "matmul_packed launch (GEMM)");
}

QMM_EXPORT size_t qmm_gemv_i8_workspace_bytes(int64_t M, int64_t K) {
  if (M <= 0 || K <= 0 || K % 32 != 0) return 0;
  return qmm::gemv_i8_workspace_bytes(M, K);
}

namespace {

// The checks qmm_gemv_i8 and qmm_gemv_i8_noalloc share, in the documented order.
int check_gemv_i8(int kind, const void *P, const void *x, int x_dtype, const float *y, int64_t M, int64_t N,
                  int64_t K) {
  int st = check_packed(kind, M, N, K);
  if (st) return st;
  if (!qmm::gemv_i8_supported(kind))
    return fail(QMM_ERR_UNSUPPORTED_KIND,
                "the int8-activation GEMV takes Q8_0, Q4_0, Q5_0, IQ4_NL or MXFP4 weights, not kind %d", kind);
  if ((st = check_dtype(x_dtype))) return st;
  if (!P || !y) return fail(QMM_ERR_BAD_ARG, "P or y is NULL");
  if (!aligned(P, 16)) return fail(QMM_ERR_BAD_ARG, "P is not 16-byte aligned");
  if ((st = check_act(x, x_dtype, "x"))) return st;
  if (!aligned(y, 4)) return fail(QMM_ERR_BAD_ARG, "y is not 4-byte aligned");
  if (M > QMM_GEMV_MAX_M) return fail(QMM_ERR_BAD_ARG, "GEMV takes 1..%d tokens, got M=%lld", QMM_GEMV_MAX_M, (long long)M);
  if (M * K > (int64_t)QMM_GEMV_I8_MAX_MK)
    return fail(QMM_ERR_BAD_ARG, "M*K=%lld exceeds %d (the block scales are staged in LDS)", (long long)(M * K),
                QMM_GEMV_I8_MAX_MK);
  return QMM_OK;
}

}  // namespace

QMM_EXPORT int qmm_gemv_i8(int kind, const void *P, const void *x, int x_dtype, float *y, int64_t M, int64_t N,
                           int64_t K, void *workspace, size_t workspace_bytes, void *stream) {
  int st = check_gemv_i8(kind, P, x, x_dtype, y, M, N, K);
  if (st) return st;
  const size_t need = qmm::gemv_i8_workspace_bytes(M, K);
  if (!workspace || workspace_bytes < need || !aligned(workspace, 256))
    return fail(QMM_ERR_WORKSPACE, "workspace needs %zu bytes (256-byte aligned), got %zu", need,
                workspace ? workspace_bytes : (size_t)0);
  return hip_status(qmm::launch_gemv_i8(kind, (const uint8_t *)P, x, x_dtype == QMM_F16, y, (int)M, N, K, workspace,
                                        (hipStream_t)stream),
                    "gemv_i8 launch");
}

QMM_EXPORT int qmm_gemv_i8_noalloc(int kind, const void *P, const void *x, int x_dtype, float *y, int64_t M,
                                   int64_t N, int64_t K, void *stream) {
  int st = check_gemv_i8(kind, P, x, x_dtype, y, M, N, K);
  if (st) return st;
  const size_t need = qmm::gemv_i8_workspace_bytes(M, K);
  if (need > (size_t)QMM_GEMV_I8_SCRATCH_BYTES)  // excluded by the M * K limit; kept as the scratch's own bound
    return fail(QMM_ERR_BAD_ARG, "M=%lld K=%lld needs %zu bytes of scratch, more than the %d the library holds",
                (long long)M, (long long)K, need, QMM_GEMV_I8_SCRATCH_BYTES);
  void *scratch = nullptr;
  hipError_t e = qmm::gemv_i8_scratch(&scratch);
  if (e != hipSuccess) return hip_status(e, "locating the gemv_i8 scratch on the current device");
  return hip_status(qmm::launch_gemv_i8(kind, (const uint8_t *)P, x, x_dtype == QMM_F16, y, (int)M, N, K, scratch,
                                        (hipStream_t)stream),
                    "gemv_i8_noalloc launch");
}

QMM_EXPORT int qmm_moe_packed(int kind, const void *P, int64_t E, const int32_t *ids, int64_t topk, const void *X,
                              int x_dtype, int x_per_slot, float *Y, int64_t M, int64_t N, int64_t K, void *workspace,
                              size_t workspace_bytes, void *stream) {
  if (E <= 0 || topk <= 0)
    return fail(QMM_ERR_EMPTY_SHAPE, "empty shape: E=%lld topk=%lld", (long long)E, (long long)topk);
  int st = check_packed(kind, M, N, K);
  if (st) return st;
  if ((st = check_dtype(x_dtype))) return st;
  if (!P || !ids || !Y) return fail(QMM_ERR_BAD_ARG, "P, ids or Y is NULL");
  if (!aligned(P, 16)) return fail(QMM_ERR_BAD_ARG, "P is not 16-byte aligned");
  if ((st = check_act(X, x_dtype, "X"))) return st;
  if (!aligned(ids, 4) || !aligned(Y, 4)) return fail(QMM_ERR_BAD_ARG, "ids or Y is not 4-byte aligned");
  if (x_per_slot != 0 && x_per_slot != 1) return fail(QMM_ERR_BAD_ARG, "x_per_slot must be 0 or 1");
  if (E > qmm::kMoeMaxExperts) return fail(QMM_ERR_BAD_ARG, "E=%lld exceeds %lld experts", (long long)E, (long long)qmm::kMoeMaxExperts);
  if (M * topk > ((int64_t)1 << 31) - 1 || M * topk * K >= ((int64_t)1 << 31))
    return fail(QMM_ERR_BAD_ARG, "M*topk*K=%lld exceeds 2^31-1", (long long)(M * topk * K));
  if (N > ((int64_t)1 << 31) / 4) return fail(QMM_ERR_BAD_ARG, "N=%lld exceeds the supported range", (long long)N);
  if (E * qmm::packed_bytes_of(kind, N, K) > ((int64_t)1 << 40))
    return fail(QMM_ERR_BAD_ARG, "E=%lld experts of N=%lld, K=%lld exceed the supported range", (long long)E,
                (long long)N, (long long)K);
  const size_t need = qmm::moe_workspace_bytes(E, M, topk);
  if (!workspace || workspace_bytes < need || !aligned(workspace, 4))
    return fail(QMM_ERR_WORKSPACE, "workspace needs %zu bytes (4-byte aligned), got %zu", need, workspace_bytes);
  return hip_status(qmm::launch_moe(kind, (const uint8_t *)P, E, ids, topk, X, x_dtype == QMM_F16, x_per_slot, Y, M,
                                    N, K, workspace, (hipStream_t)stream, true),
                    "moe_packed launch");
}

// ---------------------------------------------------------------------------
// Rotary positions, the paged key/value cache, attention over it
// ---------------------------------------------------------------------------
namespace {

bool cache_kind(int kind) { return kind == QMM_CACHE_F16 || kind == QMM_Q8_0 || kind == QMM_Q4_0; }

// Zero dimensions, kinds, head_dim against the block: the shared first checks
// of the cache calls.  `rows` is T or B.
int check_cache_shape(const qmm::KvCache &c, int64_t rows) {
  if (c.n_pages <= 0 || c.page_size <= 0 || c.n_kv <= 0 || c.head_dim <= 0 || rows <= 0)
    return fail(QMM_ERR_EMPTY_SHAPE, "empty shape: n_pages=%lld page_size=%lld n_kv=%lld head_dim=%lld rows=%lld",
                (long long)c.n_pages, (long long)c.page_size, (long long)c.n_kv, (long long)c.head_dim,
                (long long)rows);
  for (int kind : {c.k_kind, c.v_kind})
    if (!cache_kind(kind))
      return fail(QMM_ERR_UNSUPPORTED_KIND, "cache kind %d is none of F16 (%d), Q8_0 (%d), Q4_0 (%d)", kind,
                  QMM_CACHE_F16, QMM_Q8_0, QMM_Q4_0);
  if (c.head_dim % 32 != 0)
    return fail(QMM_ERR_K_NOT_BLOCK_ALIGNED, "head_dim=%lld is not a whole number of 32-element blocks",
                (long long)c.head_dim);
  return QMM_OK;
}

bool head_dim_supported(int64_t d) { return d == 64 || d == 96 || d == 128 || d == 192 || d == 256; }

int check_cache(const qmm::KvCache &c) {
  if (!head_dim_supported(c.head_dim))
    return fail(QMM_ERR_BAD_ARG, "head_dim=%lld is none of 64, 96, 128, 192, 256", (long long)c.head_dim);
  if (c.page_size % 32 != 0 || c.page_size > 65536)
    return fail(QMM_ERR_BAD_ARG, "page_size=%lld is not a multiple of 32 up to 65536", (long long)c.page_size);
  if (c.n_kv > 1024 || c.n_pages > INT32_MAX || c.n_pages * c.page_size > INT32_MAX)
    return fail(QMM_ERR_BAD_ARG, "n_kv=%lld or n_pages=%lld exceeds the supported range", (long long)c.n_kv,
                (long long)c.n_pages);
  if (!c.k_pages || !c.v_pages) return fail(QMM_ERR_BAD_ARG, "k_pages or v_pages is NULL");
  if (!aligned(c.k_pages, 16) || !aligned(c.v_pages, 16))
    return fail(QMM_ERR_BAD_ARG, "k_pages or v_pages is not 16-byte aligned");
  return QMM_OK;
}

// Rows of H heads: pointer, alignment, stride.
int check_rows(const void *x, int dtype, int64_t stride, int64_t row, int64_t T, const char *what) {
  int st = check_act(x, dtype, what);
  if (st) return st;
  if (stride < row || stride > ((int64_t)1 << 40) / T)
    return fail(QMM_ERR_BAD_ARG, "the row stride %lld of %s is below its %lld elements or out of range",
                (long long)stride, what, (long long)row);
  return QMM_OK;
}

// The rotation of q into q_out.
int check_rope(const qmm::KvWrite &w, int64_t H, int64_t D) {
  if (w.n_rot <= 0 || w.n_rot % 2 != 0 || w.n_rot > D)
    return fail(QMM_ERR_BAD_ARG, "n_rot=%lld is not an even number of elements within head_dim=%lld",
                (long long)w.n_rot, (long long)D);
  if (!w.freqs || !w.pos || !aligned(w.freqs, 8) || !aligned(w.pos, 4))
    return fail(QMM_ERR_BAD_ARG, "freqs or pos is NULL or misaligned");
  int st = check_rows(w.q, w.f16 ? QMM_F16 : QMM_F32, w.q_stride, H * D, w.T, "the rows to rotate");
  if (st) return st;
  if ((st = check_rows(w.q_out, w.q_out_f16 ? QMM_F16 : QMM_F32, w.q_out_stride, H * D, w.T, "the rotated rows")))
    return st;
  if (w.q == w.q_out && (w.f16 != w.q_out_f16 || w.q_stride != w.q_out_stride))
    return fail(QMM_ERR_BAD_ARG, "rotating in place needs equal types and strides");
  return QMM_OK;
}

int kv_write_checked(const qmm::KvCache &c, qmm::KvWrite &w, int dtype, int q_out_dtype, int layout, void *stream) {
  if (w.rope && w.n_q <= 0) return fail(QMM_ERR_EMPTY_SHAPE, "empty shape: n_q=%lld", (long long)w.n_q);
  int st = check_cache_shape(c, w.T);
  if (st) return st;
  if ((st = check_dtype(dtype))) return st;
  if (w.rope && (st = check_dtype(q_out_dtype))) return st;
  if ((st = check_cache(c))) return st;
  if (w.T > INT32_MAX || (w.rope && w.n_q > 65536) || w.T * (c.n_kv + (w.rope ? w.n_q : 0)) * c.head_dim > INT32_MAX)
    return fail(QMM_ERR_BAD_ARG, "T=%lld tokens exceed the supported range", (long long)w.T);
  const int64_t row = c.n_kv * c.head_dim;
  if ((st = check_rows(w.k, dtype, w.k_stride, row, w.T, "k"))) return st;
  if ((st = check_rows(w.v, dtype, w.v_stride, row, w.T, "v"))) return st;
  if (!w.slots || !aligned(w.slots, 4)) return fail(QMM_ERR_BAD_ARG, "slots is NULL or misaligned");
  w.f16 = dtype == QMM_F16;
  if (w.rope) {
    w.q_out_f16 = q_out_dtype == QMM_F16;
    if (layout != QMM_ROPE_HALF && layout != QMM_ROPE_INTERLEAVED)
      return fail(QMM_ERR_BAD_ARG, "layout %d is neither QMM_ROPE_HALF nor QMM_ROPE_INTERLEAVED", layout);
    w.interleaved = layout == QMM_ROPE_INTERLEAVED;
    if ((st = check_rope(w, w.n_q, c.head_dim))) return st;
  }
  return hip_status(qmm::launch_kv_write(c, w, (hipStream_t)stream), w.rope ? "kv_append launch" : "kv_write launch");
}

}  // namespace

QMM_EXPORT int64_t qmm_kv_page_bytes(int kind, int64_t page_size, int64_t n_kv, int64_t head_dim) {
  if (!cache_kind(kind) || page_size <= 0 || page_size % 32 != 0 || page_size > 65536 || n_kv <= 0 || n_kv > 1024 ||
      !head_dim_supported(head_dim))
    return -1;
  return qmm::kv_page_bytes(kind, page_size, n_kv, head_dim);
}

QMM_EXPORT int qmm_rope_freqs(double *freqs, float *mscale, int64_t n_rot, double base, const float *factors,
                              double factor, int64_t orig_ctx, double beta_fast, double beta_slow) {
  if (n_rot <= 0) return fail(QMM_ERR_EMPTY_SHAPE, "empty shape: n_rot=%lld", (long long)n_rot);
  if (n_rot % 2 != 0 || n_rot > 65536 || !freqs) return fail(QMM_ERR_BAD_ARG, "n_rot=%lld is odd or out of range, or freqs is NULL", (long long)n_rot);
  if (!(base > 1.0) || !isfinite(base)) return fail(QMM_ERR_BAD_ARG, "base=%g is not above 1", base);
  if (!(factor >= 1.0) || !isfinite(factor)) return fail(QMM_ERR_BAD_ARG, "factor=%g is not at least 1", factor);
  if (orig_ctx < 0) return fail(QMM_ERR_BAD_ARG, "orig_ctx=%lld is negative", (long long)orig_ctx);
  const bool yarn = orig_ctx > 0 && factor > 1.0;
  if (yarn && !(beta_slow > 0.0 && beta_fast > beta_slow))
    return fail(QMM_ERR_BAD_ARG, "YaRN needs beta_fast > beta_slow > 0, got %g and %g", beta_fast, beta_slow);
  for (int64_t i = 0; factors && i < n_rot / 2; ++i)
    if (!isfinite(factors[i]) || factors[i] == 0.0f)
      return fail(QMM_ERR_BAD_ARG, "factors[%lld]=%g is zero or not finite", (long long)i, (double)factors[i]);
  const double n = (double)n_rot;
  double low = 0.0, high = 1.0;
  if (yarn) {
    const double per_turn = n / (2.0 * log(base)), turns = (double)orig_ctx / (2.0 * M_PI);
    low = fmax(floor(per_turn * log(turns / beta_fast)), 0.0);
    high = fmin(ceil(per_turn * log(turns / beta_slow)), n - 1.0);
  }
  for (int64_t i = 0; i < n_rot / 2; ++i) {
    double f = pow(base, -2.0 * (double)i / n);
    if (factors) f /= (double)factors[i];
    if (yarn) {
      const double ramp = fmin(fmax(((double)i - low) / fmax(high - low, 0.001), 0.0), 1.0);
      f = f * (1.0 - ramp) + f / factor * ramp;
    } else {
      f /= factor;
    }
    freqs[i] = f;
  }
  if (mscale) *mscale = yarn ? (float)(0.1 * log(factor) + 1.0) : 1.0f;
  return ok();
}

QMM_EXPORT int qmm_rope(const double *freqs, int64_t n_rot, int layout, float mscale, const int32_t *pos,
                        const void *x, int x_dtype, int64_t x_stride, void *y, int y_dtype, int64_t y_stride,
                        int64_t T, int64_t H, int64_t head_dim, void *stream) {
  if (T <= 0 || H <= 0 || head_dim <= 0)
    return fail(QMM_ERR_EMPTY_SHAPE, "empty shape: T=%lld H=%lld head_dim=%lld", (long long)T, (long long)H,
                (long long)head_dim);
  int st = check_dtype(x_dtype);
  if (st) return st;
  if ((st = check_dtype(y_dtype))) return st;
  if (layout != QMM_ROPE_HALF && layout != QMM_ROPE_INTERLEAVED)
    return fail(QMM_ERR_BAD_ARG, "layout %d is neither QMM_ROPE_HALF nor QMM_ROPE_INTERLEAVED", layout);
  if (head_dim % 2 != 0 || head_dim > 65536 || H > 65536 || T > INT32_MAX || T * H * head_dim > (int64_t)1 << 32)
    return fail(QMM_ERR_BAD_ARG, "head_dim=%lld is odd, or T=%lld, H=%lld exceed the supported range",
                (long long)head_dim, (long long)T, (long long)H);
  qmm::KvWrite w{};
  w.q = x, w.q_stride = x_stride, w.q_out = y, w.q_out_stride = y_stride;
  w.f16 = x_dtype == QMM_F16, w.q_out_f16 = y_dtype == QMM_F16;
  w.pos = pos, w.T = T, w.n_q = H, w.freqs = freqs, w.n_rot = n_rot;
  w.interleaved = layout == QMM_ROPE_INTERLEAVED, w.mscale = mscale;
  if ((st = check_rope(w, H, head_dim))) return st;
  return hip_status(qmm::launch_rope(w, H, head_dim, (hipStream_t)stream), "rope launch");
}

QMM_EXPORT int qmm_kv_write(int k_kind, int v_kind, void *k_pages, void *v_pages, int64_t n_pages, int64_t page_size,
                            int64_t n_kv, int64_t head_dim, const void *k, int64_t k_stride, const void *v,
                            int64_t v_stride, int dtype, const int32_t *slots, int64_t T, void *stream) {
  const qmm::KvCache c{k_kind, v_kind, k_pages, v_pages, n_pages, page_size, n_kv, head_dim};
  qmm::KvWrite w{};
  w.k = k, w.v = v, w.k_stride = k_stride, w.v_stride = v_stride, w.slots = slots, w.T = T;
  return kv_write_checked(c, w, dtype, dtype, QMM_ROPE_HALF, stream);
}

QMM_EXPORT int qmm_kv_append(const double *freqs, int64_t n_rot, int layout, float mscale, const int32_t *pos,
                             const void *q, int64_t q_stride, int64_t n_q, void *q_out, int q_out_dtype,
                             int64_t q_out_stride, int k_kind, int v_kind, void *k_pages, void *v_pages,
                             int64_t n_pages, int64_t page_size, int64_t n_kv, int64_t head_dim, const void *k,
                             int64_t k_stride, const void *v, int64_t v_stride, int dtype, const int32_t *slots,
                             int64_t T, void *stream) {
  const qmm::KvCache c{k_kind, v_kind, k_pages, v_pages, n_pages, page_size, n_kv, head_dim};
  qmm::KvWrite w{};
  w.k = k, w.v = v, w.k_stride = k_stride, w.v_stride = v_stride, w.slots = slots, w.T = T;
  w.q = q, w.q_stride = q_stride, w.n_q = n_q, w.q_out = q_out, w.q_out_stride = q_out_stride;
  w.rope = 1, w.freqs = freqs, w.n_rot = n_rot, w.mscale = mscale, w.pos = pos;
  return kv_write_checked(c, w, dtype, q_out_dtype, layout, stream);
}

QMM_EXPORT int qmm_kv_read(int k_kind, int v_kind, const void *k_pages, const void *v_pages, int64_t n_pages,
                           int64_t page_size, int64_t n_kv, int64_t head_dim, const int32_t *slots, int64_t T,
                           void *k_out, void *v_out, int dtype, void *stream) {
  const qmm::KvCache c{k_kind, v_kind, (void *)k_pages, (void *)v_pages, n_pages, page_size, n_kv, head_dim};
  int st = check_cache_shape(c, T);
  if (st) return st;
  if ((st = check_dtype(dtype))) return st;
  if ((st = check_cache(c))) return st;
  if (T > INT32_MAX || T * n_kv * head_dim > INT32_MAX)
    return fail(QMM_ERR_BAD_ARG, "T=%lld tokens exceed the supported range", (long long)T);
  if (!slots || !aligned(slots, 4)) return fail(QMM_ERR_BAD_ARG, "slots is NULL or misaligned");
  if (!k_out || !v_out || !aligned(k_out, 16) || !aligned(v_out, 16))
    return fail(QMM_ERR_BAD_ARG, "k_out or v_out is NULL or not 16-byte aligned");
  return hip_status(qmm::launch_kv_read(c, slots, T, k_out, v_out, dtype == QMM_F16, (hipStream_t)stream),
                    "kv_read launch");
}

namespace {
// Largest grids (HIP: fewer than 2^32 threads) and counts of the attention
// call.
bool attn_sizes_ok(int64_t B, int64_t n_q, int64_t n_kv) {
  return B <= 65536 && n_q <= 65536 && n_kv <= 1024 && n_q % n_kv == 0 && B * n_q <= ((int64_t)1 << 23);
}
}  // namespace

QMM_EXPORT size_t qmm_attn_decode_workspace_bytes(int64_t B, int64_t n_q, int64_t n_kv, int64_t head_dim) {
  if (B <= 0 || n_q <= 0 || n_kv <= 0 || !head_dim_supported(head_dim) || !attn_sizes_ok(B, n_q, n_kv)) return 0;
  return qmm::attn_workspace_bytes(B, n_q, n_kv, head_dim);
}

QMM_EXPORT int qmm_attn_decode(int k_kind, int v_kind, const void *k_pages, const void *v_pages, int64_t n_pages,
                               int64_t page_size, int64_t n_kv, int64_t head_dim, const void *q, int dtype,
                               int64_t q_stride, int64_t n_q, const int32_t *block_table, int64_t max_pages,
                               const int32_t *seq_lens, int64_t B, float scale, int64_t window, const float *sinks,
                               void *out, void *workspace, size_t workspace_bytes, void *stream) {
  const qmm::KvCache c{k_kind, v_kind, (void *)k_pages, (void *)v_pages, n_pages, page_size, n_kv, head_dim};
  if (n_q <= 0 || max_pages <= 0)
    return fail(QMM_ERR_EMPTY_SHAPE, "empty shape: n_q=%lld max_pages=%lld", (long long)n_q, (long long)max_pages);
  int st = check_cache_shape(c, B);
  if (st) return st;
  if ((st = check_dtype(dtype))) return st;
  if ((st = check_cache(c))) return st;
  if (!attn_sizes_ok(B, n_q, n_kv))
    return fail(QMM_ERR_BAD_ARG, "n_q=%lld is not a multiple of n_kv=%lld, or they or B=%lld exceed the supported range",
                (long long)n_q, (long long)n_kv, (long long)B);
  if (max_pages > INT32_MAX || max_pages * page_size > INT32_MAX)
    return fail(QMM_ERR_BAD_ARG, "max_pages=%lld exceeds the supported range", (long long)max_pages);
  if (!isfinite(scale)) return fail(QMM_ERR_BAD_ARG, "scale is not finite");
  if (window < 0) return fail(QMM_ERR_BAD_ARG, "window=%lld is negative", (long long)window);
  if ((st = check_rows(q, dtype, q_stride, n_q * head_dim, B, "q"))) return st;
  if (!block_table || !seq_lens || !aligned(block_table, 4) || !aligned(seq_lens, 4))
    return fail(QMM_ERR_BAD_ARG, "block_table or seq_lens is NULL or misaligned");
  if (sinks && !aligned(sinks, 4)) return fail(QMM_ERR_BAD_ARG, "sinks is misaligned");
  if (!out || !aligned(out, 16)) return fail(QMM_ERR_BAD_ARG, "out is NULL or not 16-byte aligned");
  const size_t need = qmm::attn_workspace_bytes(B, n_q, n_kv, head_dim);
  if (!workspace || workspace_bytes < need || !aligned(workspace, 16))
    return fail(QMM_ERR_WORKSPACE, "workspace needs %zu bytes (16-byte aligned), got %zu", need,
                workspace ? workspace_bytes : (size_t)0);
  const qmm::AttnDecode d{q,     q_stride, dtype == QMM_F16, n_q,   B,   block_table, max_pages,
                          seq_lens, scale, window,           sinks, out, workspace};
  return hip_status(qmm::launch_attn_decode(c, d, (hipStream_t)stream), "attn_decode launch");
}

QMM_EXPORT int qmm_dequant(int kind, const void *W, float *out, int64_t n_elems, void *stream) {
  if (n_elems <= 0) return fail(QMM_ERR_EMPTY_SHAPE, "empty shape: n_elems=%lld", (long long)n_elems);
  const KindInfo *k = find_kind(kind);
  if (!k) return fail(QMM_ERR_UNSUPPORTED_KIND, "kind %d is not one of the eleven supported kinds", kind);
  if (n_elems % k->block_elems != 0)
    return fail(QMM_ERR_K_NOT_BLOCK_ALIGNED, "n_elems=%lld is not a whole number of %s blocks", (long long)n_elems, k->name);
  if (!W || !out) return fail(QMM_ERR_BAD_ARG, "W or out is NULL");
  if (!aligned(out, 4)) return fail(QMM_ERR_BAD_ARG, "out is not 4-byte aligned");
  if (n_elems > ((int64_t)1 << 40)) return fail(QMM_ERR_BAD_ARG, "n_elems exceeds the supported range");
  return hip_status(qmm::launch_dequant(kind, (const uint8_t *)W, out, n_elems / k->block_elems, (hipStream_t)stream),
                    "dequant launch");
}

QMM_EXPORT int64_t qmm_row_bytes(int kind, int64_t K) {
  const KindInfo *k = find_kind(kind);
  if (!k || K < 0 || K % k->block_elems != 0) return -1;
  return (K / k->block_elems) * k->block_bytes;
}

QMM_EXPORT int qmm_block_geometry(int kind, int *block_bytes, int *block_elems) {
  const KindInfo *k = find_kind(kind);
  if (!k) return fail(QMM_ERR_UNSUPPORTED_KIND, "kind %d is not one of the eleven supported kinds", kind);
  if (block_bytes) *block_bytes = k->block_bytes;
  if (block_elems) *block_elems = k->block_elems;
  return ok();
}

QMM_EXPORT int qmm_kind_from_name(const char *name) {
  if (!name) return -1;
  for (const KindInfo &k : kKinds)
    if (strcmp(k.name, name) == 0) return k.id;
  return -1;
}

QMM_EXPORT const char *qmm_kind_name(int kind) {
  const KindInfo *k = find_kind(kind);
  return k ? k->name : nullptr;
}

QMM_EXPORT const char *qmm_status_string(int status) {
  switch (status) {
    case QMM_OK: return "ok";
    case QMM_ERR_EMPTY_SHAPE: return "empty shape";
    case QMM_ERR_UNSUPPORTED_KIND: return "unsupported kind";
    case QMM_ERR_K_NOT_BLOCK_ALIGNED: return "K is not a whole number of blocks";
    case QMM_ERR_BAD_DTYPE: return "bad activation dtype";
    case QMM_ERR_BAD_ARG: return "bad argument";
    case QMM_ERR_HIP: return "HIP launch failed";
    case QMM_ERR_WORKSPACE: return "workspace missing or too small";
  }
  return "unknown status";
}

QMM_EXPORT const char *qmm_last_error(void) { return g_last_error.c_str(); }
