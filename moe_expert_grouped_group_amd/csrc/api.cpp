// C-ABI entry points of libmxfp8moe.so: argument validation, then kernel
// launches on the caller's stream.  Nothing here allocates, frees or
// synchronizes.  The contracts are documented in include/mxfp8moe.h.
#include "../../include/mxfp8moe.h"

#include <hip/hip_runtime.h>

#include <cstdarg>
#include <cstdio>
#include <cstring>

#include "kernels.h"
#include "ragged_common.h"

namespace {

thread_local char g_err[512] = "";

mxfp8_status fail(mxfp8_status st, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_err, sizeof(g_err), fmt, ap);
  va_end(ap);
  return st;
}

mxfp8_status ok() {
  g_err[0] = '\0';
  return MXFP8_OK;
}

mxfp8_status hip_status(hipError_t e, const char* what) {
  if (e != hipSuccess) return fail(MXFP8_EHIP, "%s: %s", what, hipGetErrorString(e));
  return ok();
}

#define REQUIRE(cond, ...)                                 \
  do {                                                     \
    if (!(cond)) return fail(MXFP8_EINVAL, __VA_ARGS__);   \
  } while (0)

// The native grouped path takes device-resident int64 splits; a host array is
// an error (mirrors the ValueError for host m_splits in "Improve device-init
// grouped linear module with single grouped weight support").
mxfp8_status check_device_splits(const int64_t* m_splits, int32_t G, const char* fn) {
  if (m_splits == nullptr) return fail(MXFP8_EINVAL, "%s: m_splits is NULL", fn);
  if (G < 1) return fail(MXFP8_EINVAL, "%s: G = %d must be >= 1", fn, (int)G);
  hipPointerAttribute_t attr;
  std::memset(&attr, 0, sizeof(attr));
  const hipError_t e = hipPointerGetAttributes(&attr, m_splits);
  if (e != hipSuccess) {
    (void)hipGetLastError();  // clear the sticky error of the failed query
    return fail(MXFP8_EINVAL,
                "%s: m_splits must be a device int64 array (pointer query failed: %s)", fn,
                hipGetErrorString(e));
  }
  if (attr.type != hipMemoryTypeDevice && attr.type != hipMemoryTypeManaged)
    return fail(MXFP8_EINVAL, "%s: m_splits must be a device int64 array, got a host pointer",
                fn);
  return MXFP8_OK;
}

hipStream_t as_stream(void* s) { return reinterpret_cast<hipStream_t>(s); }

}  // namespace

extern "C" {

const char* mxfp8_last_error(void) { return g_err; }

int32_t mxfp8_abi_version(void) { return 6; }

size_t mxfp8_dbias_workspace_bytes(int64_t T, int64_t N) {
  if (T <= 0 || N <= 0) return 0;
  return (size_t)((T + 127) / 128) * (size_t)N * sizeof(float);
}

mxfp8_status mxfp8_group_quantize(const uint16_t* x, int64_t T, int64_t K, uint32_t usage,
                                  uint8_t* q_row, uint8_t* s_row, uint8_t* q_col,
                                  uint8_t* s_col, const int32_t* noop_flag, void* stream) {
  const char* fn = "mxfp8_group_quantize";
  REQUIRE(x != nullptr || T == 0, "%s: x is NULL", fn);
  REQUIRE(usage != 0 && (usage & ~(MXFP8_ROWWISE | MXFP8_COLWISE)) == 0,
          "%s: usage must be a non-empty combination of MXFP8_ROWWISE and MXFP8_COLWISE", fn);
  REQUIRE(T >= 0 && T % 128 == 0, "%s: T = %lld must be a multiple of 128", fn, (long long)T);
  REQUIRE(K > 0 && K % 512 == 0, "%s: K = %lld must be a positive multiple of 512", fn,
          (long long)K);
  if (T == 0) return ok();   // nothing to read or write: every buffer is empty
  const bool row = usage & MXFP8_ROWWISE, col = usage & MXFP8_COLWISE;
  REQUIRE(!row || (q_row && s_row), "%s: ROWWISE requested but q_row/s_row is NULL", fn);
  REQUIRE(!col || (q_col && s_col), "%s: COLWISE requested but q_col/s_col is NULL", fn);
  hipError_t e;
  if (col)
    e = mx::launch_quant_rowcol(x, T, K, row ? q_row : nullptr, row ? s_row : nullptr, q_col,
                                s_col, noop_flag, as_stream(stream));
  else
    e = mx::launch_quant_rowwise(x, T, K, q_row, s_row, noop_flag, as_stream(stream));
  return hip_status(e, fn);
}

mxfp8_status mxfp8_requant_colwise(const uint8_t* q_row, const uint8_t* s_row, int64_t T,
                                   int64_t K, uint8_t* q_col, uint8_t* s_col,
                                   const int64_t* m_splits, int32_t G, float* dbias,
                                   void* workspace, size_t workspace_bytes, void* stream) {
  const char* fn = "mxfp8_requant_colwise";
  REQUIRE(T == 0 || (q_row && s_row && q_col && s_col), "%s: NULL data/scale pointer", fn);
  REQUIRE(T >= 0 && T % 128 == 0, "%s: T = %lld must be a multiple of 128", fn, (long long)T);
  REQUIRE(K > 0 && K % 512 == 0, "%s: K = %lld must be a positive multiple of 512", fn,
          (long long)K);
  float* partial = nullptr;
  if (dbias != nullptr) {
    mxfp8_status st = check_device_splits(m_splits, G, fn);
    if (st != MXFP8_OK) return st;
    REQUIRE((workspace != nullptr || T == 0) &&
                workspace_bytes >= mxfp8_dbias_workspace_bytes(T, K),
            "%s: dbias needs a workspace of %zu bytes", fn, mxfp8_dbias_workspace_bytes(T, K));
    partial = static_cast<float*>(workspace);
  }
  hipStream_t st = as_stream(stream);
  hipError_t e = hipSuccess;
  if (T > 0) e = mx::launch_requant_colwise(q_row, s_row, T, K, q_col, s_col, partial, st);
  if (e == hipSuccess && dbias != nullptr)
    e = mx::launch_dbias_finalize(partial, m_splits, G, T, K, dbias, st);
  return hip_status(e, fn);
}

mxfp8_status mxfp8_group_quantize_requant(const uint16_t* x, int64_t T, int64_t K,
                                          uint8_t* q_row, uint8_t* s_row, uint8_t* q_col,
                                          uint8_t* s_col, const int64_t* m_splits, int32_t G,
                                          float* dbias, void* workspace, size_t workspace_bytes,
                                          void* stream) {
  const char* fn = "mxfp8_group_quantize_requant";
  REQUIRE(T == 0 || (x && q_row && s_row && q_col && s_col), "%s: NULL data/scale pointer", fn);
  REQUIRE(T >= 0 && T % 128 == 0, "%s: T = %lld must be a multiple of 128", fn, (long long)T);
  REQUIRE(K > 0 && K % 512 == 0, "%s: K = %lld must be a positive multiple of 512", fn,
          (long long)K);
  float* partial = nullptr;
  if (dbias != nullptr) {
    mxfp8_status st = check_device_splits(m_splits, G, fn);
    if (st != MXFP8_OK) return st;
    REQUIRE((workspace != nullptr || T == 0) &&
                workspace_bytes >= mxfp8_dbias_workspace_bytes(T, K),
            "%s: dbias needs a workspace of %zu bytes", fn, mxfp8_dbias_workspace_bytes(T, K));
    partial = static_cast<float*>(workspace);
  }
  hipStream_t st = as_stream(stream);
  hipError_t e = hipSuccess;
  if (T > 0) e = mx::launch_quant_row_requant(x, T, K, q_row, s_row, q_col, s_col, partial, st);
  if (e == hipSuccess && dbias != nullptr)
    e = mx::launch_dbias_finalize(partial, m_splits, G, T, K, dbias, st);
  return hip_status(e, fn);
}

mxfp8_status mxfp8_group_quantize_requant_noalloc(const uint16_t* x, int64_t T, int64_t K,
                                                  uint8_t* q_row, uint8_t* s_row, uint8_t* q_col,
                                                  uint8_t* s_col, const int64_t* m_splits,
                                                  int32_t G, float* dbias, void* stream) {
  const char* fn = "mxfp8_group_quantize_requant_noalloc";
  REQUIRE(T == 0 || (x && q_row && s_row && q_col && s_col), "%s: NULL data/scale pointer", fn);
  REQUIRE(T >= 0 && T % 128 == 0, "%s: T = %lld must be a multiple of 128", fn, (long long)T);
  REQUIRE(K > 0 && K % 512 == 0, "%s: K = %lld must be a positive multiple of 512", fn,
          (long long)K);
  float* partial = nullptr;
  if (dbias != nullptr) {
    const size_t need = mxfp8_dbias_workspace_bytes(T, K);
    REQUIRE(need <= mx::noalloc_scratch_bytes(),
            "%s: dbias of a [%lld, %lld] operand needs %zu bytes of partial sums, more than the "
            "%zu-byte static scratch (MXFP8_NOALLOC_SCRATCH_BYTES); use "
            "mxfp8_group_quantize_requant with a workspace",
            fn, (long long)T, (long long)K, need, mx::noalloc_scratch_bytes());
    mxfp8_status st = check_device_splits(m_splits, G, fn);
    if (st != MXFP8_OK) return st;
    if (T > 0) {
      const hipError_t e = mx::noalloc_scratch(&partial);
      if (e != hipSuccess) return hip_status(e, fn);
    }
  }
  hipStream_t st = as_stream(stream);
  hipError_t e = hipSuccess;
  if (T > 0) e = mx::launch_quant_row_requant(x, T, K, q_row, s_row, q_col, s_col, partial, st);
  if (e == hipSuccess && dbias != nullptr)
    e = mx::launch_dbias_finalize(partial, m_splits, G, T, K, dbias, st);
  return hip_status(e, fn);
}

mxfp8_status mxfp8_grouped_dbias(const uint8_t* q_row, const uint8_t* s_row, int64_t T,
                                 int64_t N, const int64_t* m_splits, int32_t G, float* dbias,
                                 void* workspace, size_t workspace_bytes, void* stream) {
  const char* fn = "mxfp8_grouped_dbias";
  REQUIRE(dbias && (T == 0 || (q_row && s_row)), "%s: NULL pointer", fn);
  REQUIRE(T >= 0 && T % 128 == 0, "%s: T = %lld must be a multiple of 128", fn, (long long)T);
  REQUIRE(N > 0 && N % 512 == 0, "%s: N = %lld must be a positive multiple of 512", fn,
          (long long)N);
  mxfp8_status s = check_device_splits(m_splits, G, fn);
  if (s != MXFP8_OK) return s;
  REQUIRE((workspace != nullptr || T == 0) &&
              workspace_bytes >= mxfp8_dbias_workspace_bytes(T, N),
          "%s: needs a workspace of %zu bytes", fn, mxfp8_dbias_workspace_bytes(T, N));
  float* partial = static_cast<float*>(workspace);
  hipStream_t st = as_stream(stream);
  hipError_t e = hipSuccess;
  if (T > 0) e = mx::launch_dbias_partial(q_row, s_row, T, N, partial, st);
  if (e == hipSuccess) e = mx::launch_dbias_finalize(partial, m_splits, G, T, N, dbias, st);
  return hip_status(e, fn);
}

size_t mxfp8_scaled_bias_workspace_bytes(int64_t T, int64_t N) {
  if (T <= 0 || N <= 0) return 0;
  return mx::scaled_bias_workspace_bytes(T, N);
}

mxfp8_status mxfp8_grouped_scaled_bias_grad(const uint8_t* q_row, const uint8_t* s_row,
                                            int64_t T, int64_t N, const int64_t* m_splits,
                                            int32_t G, const float* scales, const float* bias,
                                            float* dbias, float* dscales, void* workspace,
                                            size_t workspace_bytes, void* stream) {
  const char* fn = "mxfp8_grouped_scaled_bias_grad";
  REQUIRE(T == 0 || (q_row && s_row), "%s: NULL data/scale pointer", fn);
  REQUIRE(dbias || dscales, "%s: neither dbias nor dscales requested", fn);
  REQUIRE(!dbias || scales || T == 0, "%s: dbias needs the routing scales", fn);
  REQUIRE(!dscales || bias || T == 0, "%s: dscales needs the bias", fn);
  REQUIRE(T >= 0 && T % 128 == 0, "%s: T = %lld must be a multiple of 128", fn, (long long)T);
  REQUIRE(N > 0 && N % 512 == 0, "%s: N = %lld must be a positive multiple of 512", fn,
          (long long)N);
  mxfp8_status s = check_device_splits(m_splits, G, fn);
  if (s != MXFP8_OK) return s;
  if (T == 0) {
    // no rows: dbias is zero for every expert, dscales is empty
    if (dbias != nullptr)
      return hip_status(mx::launch_dbias_finalize(nullptr, m_splits, G, 0, N, dbias,
                                                  as_stream(stream)), fn);
    return ok();
  }
  REQUIRE(workspace != nullptr && workspace_bytes >= mx::scaled_bias_workspace_bytes(T, N),
          "%s: needs a workspace of %zu bytes", fn, mx::scaled_bias_workspace_bytes(T, N));
  return hip_status(mx::launch_scaled_bias_grad(q_row, s_row, T, N, m_splits, G, scales, bias,
                                                dbias, dscales, workspace, as_stream(stream)),
                    fn);
}

static mxfp8_status grouped_gemm_impl(const char* fn, int32_t layout, const uint8_t* a_data,
                                      const uint8_t* a_scale, const uint8_t* b_data,
                                      const uint8_t* b_scale, void* c, int32_t c_dtype, int64_t T,
                                      int64_t N, int64_t K, const int64_t* m_splits, int32_t G,
                                      int32_t* queue, void* stream) {
  REQUIRE(layout == MXFP8_LAYOUT_NT || layout == MXFP8_LAYOUT_NN || layout == MXFP8_LAYOUT_TN,
          "%s: layout %d is not NT(0), NN(1) or TN(2)", fn, (int)layout);
  if (c_dtype != MXFP8_OUT_F32 && c_dtype != MXFP8_OUT_BF16)
    return fail(MXFP8_ENOTSUP, "%s: output dtype %d is not supported (f32 = 0, bf16 = 1)", fn,
                (int)c_dtype);
  // with no tokens nothing is read, and the forward/dgrad output is empty too
  REQUIRE(T == 0 || (a_data && a_scale && b_data && b_scale && c), "%s: NULL operand pointer",
          fn);
  REQUIRE(c || layout != MXFP8_LAYOUT_TN, "%s: NULL output", fn);
  REQUIRE(T >= 0 && T % 128 == 0, "%s: T = %lld must be a multiple of 128", fn, (long long)T);
  REQUIRE(N > 0 && N % 512 == 0, "%s: N = %lld must be a positive multiple of 512", fn,
          (long long)N);
  REQUIRE(K > 0 && K % 512 == 0, "%s: K = %lld must be a positive multiple of 512", fn,
          (long long)K);
  REQUIRE(G <= 1024, "%s: G = %d exceeds the supported 1024 experts", fn, (int)G);
  mxfp8_status s = check_device_splits(m_splits, G, fn);
  if (s != MXFP8_OK) return s;
  if (T == 0 && layout != MXFP8_LAYOUT_TN) return ok();
  const hipError_t e = mx::launch_grouped_gemm(layout, a_data, a_scale, b_data, b_scale, c,
                                               c_dtype == MXFP8_OUT_BF16, T, N, K, m_splits, G,
                                               false, as_stream(stream), queue);
  return hip_status(e, fn);
}

mxfp8_status mxfp8_grouped_gemm_swiglu_quantize(const uint8_t* a_data, const uint8_t* a_scale,
                                                const uint8_t* b_data, const uint8_t* b_scale,
                                                uint16_t* h, int64_t T, int64_t F, int64_t K,
                                                const int64_t* m_splits, int32_t G,
                                                uint32_t usage, uint8_t* q_row, uint8_t* s_row,
                                                uint8_t* q_col, uint8_t* s_col, void* stream) {
  const char* fn = "mxfp8_grouped_gemm_swiglu_quantize";
  REQUIRE(usage != 0 && (usage & ~(MXFP8_ROWWISE | MXFP8_COLWISE)) == 0,
          "%s: usage must be a non-empty combination of MXFP8_ROWWISE and MXFP8_COLWISE", fn);
  REQUIRE(T >= 0 && T % 128 == 0, "%s: T = %lld must be a multiple of 128", fn, (long long)T);
  REQUIRE(F > 0 && F % 512 == 0, "%s: F = %lld must be a positive multiple of 512", fn,
          (long long)F);
  REQUIRE(K > 0 && K % 512 == 0, "%s: K = %lld must be a positive multiple of 512", fn,
          (long long)K);
  REQUIRE(G <= 1024, "%s: G = %d exceeds the supported 1024 experts", fn, (int)G);
  if (T > 0) {
    REQUIRE(a_data && a_scale && b_data && b_scale && h, "%s: NULL operand pointer", fn);
    const bool row = usage & MXFP8_ROWWISE, col = usage & MXFP8_COLWISE;
    REQUIRE(!row || (q_row && s_row), "%s: ROWWISE requested but q_row/s_row is NULL", fn);
    REQUIRE(!col || (q_col && s_col), "%s: COLWISE requested but q_col/s_col is NULL", fn);
  }
  mxfp8_status s = check_device_splits(m_splits, G, fn);
  if (s != MXFP8_OK) return s;
  if (T == 0) return ok();   // no rows: every output is empty
  const bool row = usage & MXFP8_ROWWISE, col = usage & MXFP8_COLWISE;
  return hip_status(mx::launch_grouped_gemm_swiglu(a_data, a_scale, b_data, b_scale, h, T, F, K,
                                                   m_splits, G, row ? q_row : nullptr,
                                                   row ? s_row : nullptr, col ? q_col : nullptr,
                                                   col ? s_col : nullptr, as_stream(stream)),
                    fn);
}

static mxfp8_status wgrad_accumulate_impl(const char* fn, const uint8_t* a_data,
                                          const uint8_t* a_scale, const uint8_t* b_data,
                                          const uint8_t* b_scale, float* main_grad, int64_t T,
                                          int64_t N, int64_t K, const int64_t* m_splits,
                                          int32_t G, int32_t* queue, void* stream) {
  REQUIRE(main_grad && (T == 0 || (a_data && a_scale && b_data && b_scale)), "%s: NULL pointer",
          fn);
  REQUIRE(T >= 0 && T % 128 == 0, "%s: T = %lld must be a multiple of 128", fn, (long long)T);
  REQUIRE(N > 0 && N % 512 == 0, "%s: N = %lld must be a positive multiple of 512", fn,
          (long long)N);
  REQUIRE(K > 0 && K % 512 == 0, "%s: K = %lld must be a positive multiple of 512", fn,
          (long long)K);
  REQUIRE(G <= 1024, "%s: G = %d exceeds the supported 1024 experts", fn, (int)G);
  mxfp8_status s = check_device_splits(m_splits, G, fn);
  if (s != MXFP8_OK) return s;
  if (T == 0) return ok();   // every expert is empty: main_grad stays as it is
  const hipError_t e =
      mx::launch_grouped_gemm(MXFP8_LAYOUT_TN, a_data, a_scale, b_data, b_scale, main_grad, false,
                              T, N, K, m_splits, G, true, as_stream(stream), queue);
  return hip_status(e, fn);
}

// A workspace must hold the tile counter: at least mxfp8_grouped_gemm_workspace_bytes().
static mxfp8_status check_gemm_workspace(const char* fn, void* workspace, size_t bytes) {
  REQUIRE(workspace != nullptr && bytes >= mxfp8_grouped_gemm_workspace_bytes(),
          "%s: needs a device workspace of %zu bytes", fn, mxfp8_grouped_gemm_workspace_bytes());
  return MXFP8_OK;
}

size_t mxfp8_grouped_gemm_workspace_bytes(void) { return 256; }

mxfp8_status mxfp8_grouped_gemm(int32_t layout, const uint8_t* a_data, const uint8_t* a_scale,
                                const uint8_t* b_data, const uint8_t* b_scale, void* c,
                                int32_t c_dtype, int64_t T, int64_t N, int64_t K,
                                const int64_t* m_splits, int32_t G, void* stream) {
  return grouped_gemm_impl("mxfp8_grouped_gemm", layout, a_data, a_scale, b_data, b_scale, c,
                           c_dtype, T, N, K, m_splits, G, nullptr, stream);
}

mxfp8_status mxfp8_grouped_gemm_ws(int32_t layout, const uint8_t* a_data, const uint8_t* a_scale,
                                   const uint8_t* b_data, const uint8_t* b_scale, void* c,
                                   int32_t c_dtype, int64_t T, int64_t N, int64_t K,
                                   const int64_t* m_splits, int32_t G, void* workspace,
                                   size_t workspace_bytes, void* stream) {
  const char* fn = "mxfp8_grouped_gemm_ws";
  const mxfp8_status s = check_gemm_workspace(fn, workspace, workspace_bytes);
  if (s != MXFP8_OK) return s;
  return grouped_gemm_impl(fn, layout, a_data, a_scale, b_data, b_scale, c, c_dtype, T, N, K,
                           m_splits, G, static_cast<int32_t*>(workspace), stream);
}

mxfp8_status mxfp8_grouped_gemm_wgrad_accumulate(const uint8_t* a_data, const uint8_t* a_scale,
                                                 const uint8_t* b_data, const uint8_t* b_scale,
                                                 float* main_grad, int64_t T, int64_t N, int64_t K,
                                                 const int64_t* m_splits, int32_t G,
                                                 void* stream) {
  return wgrad_accumulate_impl("mxfp8_grouped_gemm_wgrad_accumulate", a_data, a_scale, b_data,
                               b_scale, main_grad, T, N, K, m_splits, G, nullptr, stream);
}

mxfp8_status mxfp8_grouped_gemm_wgrad_accumulate_ws(const uint8_t* a_data,
                                                    const uint8_t* a_scale, const uint8_t* b_data,
                                                    const uint8_t* b_scale, float* main_grad,
                                                    int64_t T, int64_t N, int64_t K,
                                                    const int64_t* m_splits, int32_t G,
                                                    void* workspace, size_t workspace_bytes,
                                                    void* stream) {
  const char* fn = "mxfp8_grouped_gemm_wgrad_accumulate_ws";
  const mxfp8_status s = check_gemm_workspace(fn, workspace, workspace_bytes);
  if (s != MXFP8_OK) return s;
  return wgrad_accumulate_impl(fn, a_data, a_scale, b_data, b_scale, main_grad, T, N, K, m_splits,
                               G, static_cast<int32_t*>(workspace), stream);
}

mxfp8_status mxfp8_validate_splits(const int64_t* m_splits, int32_t G, int64_t T, int32_t* flag,
                                   void* stream) {
  const char* fn = "mxfp8_validate_splits";
  REQUIRE(flag != nullptr, "%s: flag is NULL", fn);
  REQUIRE(G <= 1 << 20, "%s: G = %d is too large", fn, (int)G);
  mxfp8_status s = check_device_splits(m_splits, G, fn);
  if (s != MXFP8_OK) return s;
  return hip_status(mx::launch_validate_splits(m_splits, G, T, flag, as_stream(stream)), fn);
}

mxfp8_status mxfp8_swiglu_fwd(const uint16_t* h, int64_t T, int64_t F, uint16_t* a,
                              void* stream) {
  const char* fn = "mxfp8_swiglu_fwd";
  REQUIRE(T == 0 || (h && a), "%s: NULL pointer", fn);
  REQUIRE(T >= 0, "%s: T < 0", fn);
  REQUIRE(F > 0 && F % 8 == 0, "%s: F = %lld must be a positive multiple of 8", fn, (long long)F);
  if (T == 0) return ok();
  return hip_status(mx::launch_swiglu_fwd(h, T, F, a, as_stream(stream)), fn);
}

mxfp8_status mxfp8_swiglu_quantize(const uint16_t* h, int64_t T, int64_t F, uint32_t usage,
                                   uint8_t* q_row, uint8_t* s_row, uint8_t* q_col,
                                   uint8_t* s_col, void* stream) {
  const char* fn = "mxfp8_swiglu_quantize";
  REQUIRE(h != nullptr || T == 0, "%s: h is NULL", fn);
  REQUIRE(usage != 0 && (usage & ~(MXFP8_ROWWISE | MXFP8_COLWISE)) == 0,
          "%s: usage must be a non-empty combination of MXFP8_ROWWISE and MXFP8_COLWISE", fn);
  REQUIRE(T >= 0 && T % 128 == 0, "%s: T = %lld must be a multiple of 128", fn, (long long)T);
  REQUIRE(F > 0 && F % 512 == 0, "%s: F = %lld must be a positive multiple of 512", fn,
          (long long)F);
  if (T == 0) return ok();   // nothing to read or write: every buffer is empty
  const bool row = usage & MXFP8_ROWWISE, col = usage & MXFP8_COLWISE;
  REQUIRE(!row || (q_row && s_row), "%s: ROWWISE requested but q_row/s_row is NULL", fn);
  REQUIRE(!col || (q_col && s_col), "%s: COLWISE requested but q_col/s_col is NULL", fn);
  return hip_status(mx::launch_swiglu_quant(h, T, F, row ? q_row : nullptr, row ? s_row : nullptr,
                                            col ? q_col : nullptr, col ? s_col : nullptr,
                                            as_stream(stream)),
                    fn);
}

mxfp8_status mxfp8_swiglu_bwd(const uint16_t* h, const uint16_t* da, int64_t T, int64_t F,
                              uint16_t* dh, void* stream) {
  const char* fn = "mxfp8_swiglu_bwd";
  REQUIRE(T == 0 || (h && da && dh), "%s: NULL pointer", fn);
  REQUIRE(T >= 0, "%s: T < 0", fn);
  REQUIRE(F > 0 && F % 8 == 0, "%s: F = %lld must be a positive multiple of 8", fn, (long long)F);
  if (T == 0) return ok();
  return hip_status(mx::launch_swiglu_bwd(h, da, T, F, dh, as_stream(stream)), fn);
}

mxfp8_status mxfp8_swiglu_bwd_quantize(const uint16_t* h, const uint16_t* da, int64_t T,
                                       int64_t F, uint8_t* q_row, uint8_t* s_row, uint8_t* q_col,
                                       uint8_t* s_col, const int64_t* m_splits, int32_t G,
                                       float* dbias, void* workspace, size_t workspace_bytes,
                                       void* stream) {
  const char* fn = "mxfp8_swiglu_bwd_quantize";
  REQUIRE(T == 0 || (h && da && q_row && s_row && q_col && s_col), "%s: NULL pointer", fn);
  REQUIRE(T >= 0 && T % 128 == 0, "%s: T = %lld must be a multiple of 128", fn, (long long)T);
  REQUIRE(F > 0 && F % 256 == 0, "%s: F = %lld must be a positive multiple of 256", fn,
          (long long)F);
  const int64_t K = 2 * F;
  float* partial = nullptr;
  if (dbias != nullptr) {
    mxfp8_status st = check_device_splits(m_splits, G, fn);
    if (st != MXFP8_OK) return st;
    REQUIRE((workspace != nullptr || T == 0) &&
                workspace_bytes >= mxfp8_dbias_workspace_bytes(T, K),
            "%s: dbias needs a workspace of %zu bytes", fn, mxfp8_dbias_workspace_bytes(T, K));
    partial = static_cast<float*>(workspace);
  }
  hipStream_t st = as_stream(stream);
  hipError_t e = hipSuccess;
  if (T > 0)
    e = mx::launch_swiglu_bwd_quant(h, da, T, F, q_row, s_row, q_col, s_col, partial, st);
  if (e == hipSuccess && dbias != nullptr)
    e = mx::launch_dbias_finalize(partial, m_splits, G, T, K, dbias, st);
  return hip_status(e, fn);
}

size_t mxfp8_convert_sweep_bytes(int32_t mode) { return mx::convert_sweep_bytes(mode); }

mxfp8_status mxfp8_convert_sweep(int32_t mode, void* out, size_t out_bytes, void* stream) {
  const char* fn = "mxfp8_convert_sweep";
  const size_t need = mx::convert_sweep_bytes(mode);
  REQUIRE(need != 0, "%s: unknown mode %d", fn, (int)mode);
  REQUIRE(out != nullptr && out_bytes >= need, "%s: mode %d needs a buffer of %zu bytes", fn,
          (int)mode, need);
  return hip_status(mx::launch_convert_sweep(mode, static_cast<uint8_t*>(out), as_stream(stream)),
                    fn);
}

namespace {

constexpr int64_t kI32Max = 0x7FFFFFFF;

// What the ragged products check alike: sizes, splits, and the row index.
mxfp8_status check_ragged(const char* fn, int layout, int64_t R, int64_t S, int64_t N, int64_t K,
                          const int64_t* m_splits, int32_t G, const int32_t* row_index) {
  REQUIRE(R >= 0 && S >= 0 && R <= kI32Max && S <= kI32Max,
          "%s: R = %lld and S = %lld must be 0 to 2^31 - 1", fn, (long long)R, (long long)S);
  REQUIRE(N >= 1 && K >= 1 && N <= kI32Max && K <= kI32Max,
          "%s: N = %lld and K = %lld must be 1 to 2^31 - 1", fn, (long long)N, (long long)K);
  REQUIRE(G >= 1 && G <= mx::kRaggedMaxGroups, "%s: G = %d must be 1 to %d", fn, (int)G,
          mx::kRaggedMaxGroups);
  REQUIRE(row_index == nullptr || layout != MXFP8_LAYOUT_NN, "%s: NN takes no row_index", fn);
  REQUIRE(row_index != nullptr || S == R, "%s: S = %lld must be R = %lld without a row_index", fn,
          (long long)S, (long long)R);
  REQUIRE(mx::ragged_blocks(layout, R, N, K, G) <= kI32Max, "%s: over 2^31 - 1 output tiles", fn);
  return check_device_splits(m_splits, G, fn);
}

bool aligned_to(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

void* usable_workspace(void* ws) { return aligned_to(ws, 16) ? ws : nullptr; }

}  // namespace

size_t mxfp8_ragged_gemm_workspace_bytes(int32_t layout, int32_t elem_bytes, int64_t R, int64_t S,
                                         int64_t N, int64_t K, int32_t G) {
  if (layout < 0 || layout > 2 || (elem_bytes != 1 && elem_bytes != 2) || R < 0 || S < 0 || N < 1 ||
      K < 1 || G < 1 || G > mx::kRaggedMaxGroups || R > kI32Max || S > kI32Max || N > kI32Max ||
      K > kI32Max)
    return 0;
  return mx::ragged_workspace_bytes(layout, elem_bytes, R, S, N, K, G);
}

mxfp8_status mxfp8_ragged_gemm(int32_t layout, int32_t type, const void* a, int64_t lda,
                               const void* b, int64_t ldb, void* c, int64_t ldc, int32_t c_type,
                               int64_t R, int64_t S, int64_t N, int64_t K,
                               const int64_t* m_splits, int32_t G, const int32_t* row_index,
                               void* workspace, size_t workspace_bytes, void* stream) {
  const char* fn = "mxfp8_ragged_gemm";
  REQUIRE(layout == MXFP8_LAYOUT_NT || layout == MXFP8_LAYOUT_NN || layout == MXFP8_LAYOUT_TN,
          "%s: unknown layout %d", fn, (int)layout);
  if (type != MXFP8_TYPE_BF16 && type != MXFP8_TYPE_F16)
    return fail(MXFP8_ENOTSUP, "%s: operand type %d is not supported", fn, (int)type);
  if (c_type != MXFP8_TYPE_F32 && c_type != type)
    return fail(MXFP8_ENOTSUP, "%s: output type %d is not supported", fn, (int)c_type);
  mxfp8_status st = check_ragged(fn, layout, R, S, N, K, m_splits, G, row_index);
  if (st != MXFP8_OK) return st;
  const bool tn = layout == MXFP8_LAYOUT_TN;
  REQUIRE(lda >= (layout == MXFP8_LAYOUT_NT ? K : N), "%s: lda = %lld is shorter than a row", fn,
          (long long)lda);
  REQUIRE(!tn || ldb >= K, "%s: ldb = %lld is shorter than a row", fn, (long long)ldb);
  REQUIRE(tn || ldc >= (layout == MXFP8_LAYOUT_NT ? N : K), "%s: ldc = %lld is shorter than a row",
          fn, (long long)ldc);
  if (R == 0 && !tn) return ok();
  REQUIRE(c != nullptr, "%s: c is NULL", fn);
  REQUIRE(tn ? (R == 0 || a) && (S == 0 || R == 0 || b) : b && (a || S == 0),
          "%s: NULL operand", fn);
  REQUIRE(aligned_to(a, 2) && aligned_to(b, 2) && aligned_to(c, c_type == 0 ? 4 : 2) &&
              aligned_to(row_index, 4) && aligned_to(m_splits, 8),
          "%s: a pointer is not aligned to its element", fn);
  mx::RaggedArgs p{};
  p.a = a;
  p.b = b;
  p.c = c;
  p.lda = lda;
  p.ldb = tn ? ldb : K;
  p.ldc = tn ? K : ldc;
  p.R = R;
  p.S = S;
  p.N = N;
  p.K = K;
  p.m_splits = m_splits;
  p.row_index = row_index;
  p.G = G;
  p.ws = usable_workspace(workspace);
  return hip_status(
      mx::launch_ragged_gemm(layout, type == MXFP8_TYPE_F16, c_type, p,
                             p.ws != nullptr ? workspace_bytes : 0, as_stream(stream)),
      fn);
}

size_t mxfp8_ragged_gemm_swiglu_workspace_bytes(int32_t backward, int64_t R, int64_t F, int64_t C,
                                                int32_t G) {
  if (R < 0 || F < 1 || C < 1 || G < 1 || G > mx::kRaggedMaxGroups || R > kI32Max ||
      F > kI32Max / 2 || C > kI32Max)
    return 0;
  return backward ? mx::ragged_gated_workspace_bytes(true, R, C, F, G)
                  : mx::ragged_gated_workspace_bytes(false, R, 2 * F, C, G);
}

mxfp8_status mxfp8_ragged_gemm_swiglu(int32_t type, const void* x, int64_t ldx, const void* w, void* a,
                                      int64_t lda, void* h, int64_t R, int64_t S, int64_t F, int64_t K,
                                      const int64_t* m_splits, int32_t G, const int32_t* row_index,
                                      void* workspace, size_t workspace_bytes, void* stream) {
  const char* fn = "mxfp8_ragged_gemm_swiglu";
  if (type != MXFP8_TYPE_BF16 && type != MXFP8_TYPE_F16)
    return fail(MXFP8_ENOTSUP, "%s: operand type %d is not supported", fn, (int)type);
  REQUIRE(F >= 1 && F <= kI32Max / 2, "%s: F = %lld must be 1 to 2^30 - 1", fn, (long long)F);
  mxfp8_status st = check_ragged(fn, MXFP8_LAYOUT_NT, R, S, 2 * F, K, m_splits, G, row_index);
  if (st != MXFP8_OK) return st;
  REQUIRE(ldx >= K, "%s: ldx = %lld is shorter than a row", fn, (long long)ldx);
  REQUIRE(lda >= F, "%s: lda = %lld is shorter than a row", fn, (long long)lda);
  if (R == 0) return ok();
  REQUIRE(a && w && (x || S == 0), "%s: NULL pointer", fn);
  REQUIRE(aligned_to(x, 2) && aligned_to(w, 2) && aligned_to(a, 2) && aligned_to(h, 2) &&
              aligned_to(row_index, 4) && aligned_to(m_splits, 8),
          "%s: a pointer is not aligned to its element", fn);
  mx::RaggedArgs p{};
  p.a = x;
  p.b = w;
  p.c = a;
  p.h = h;
  p.lda = ldx;
  p.ldb = K;
  p.ldc = lda;
  p.R = R;
  p.S = S;
  p.N = 2 * F;
  p.K = K;
  p.m_splits = m_splits;
  p.row_index = row_index;
  p.G = G;
  p.ws = usable_workspace(workspace);
  return hip_status(mx::launch_ragged_gated(type == MXFP8_TYPE_F16, p, p.ws != nullptr ? workspace_bytes : 0,
                                            as_stream(stream)),
                    fn);
}

mxfp8_status mxfp8_ragged_gemm_swiglu_bwd(int32_t type, const void* dy, int64_t lddy, const void* w,
                                          const void* h, void* dh, void* a, int64_t R, int64_t N,
                                          int64_t F, const int64_t* m_splits, int32_t G, void* workspace,
                                          size_t workspace_bytes, void* stream) {
  const char* fn = "mxfp8_ragged_gemm_swiglu_bwd";
  if (type != MXFP8_TYPE_BF16 && type != MXFP8_TYPE_F16)
    return fail(MXFP8_ENOTSUP, "%s: operand type %d is not supported", fn, (int)type);
  REQUIRE(F >= 1 && F <= kI32Max / 2, "%s: F = %lld must be 1 to 2^30 - 1", fn, (long long)F);
  mxfp8_status st = check_ragged(fn, MXFP8_LAYOUT_NN, R, R, N, F, m_splits, G, nullptr);
  if (st != MXFP8_OK) return st;
  REQUIRE(lddy >= N, "%s: lddy = %lld is shorter than a row", fn, (long long)lddy);
  if (R == 0) return ok();
  REQUIRE(dy && w && h && dh, "%s: NULL pointer", fn);
  REQUIRE(aligned_to(dy, 2) && aligned_to(w, 2) && aligned_to(h, 2) && aligned_to(dh, 2) &&
              aligned_to(a, 2) && aligned_to(m_splits, 8),
          "%s: a pointer is not aligned to its element", fn);
  mx::RaggedArgs p{};
  p.a = dy;
  p.b = w;
  p.c = dh;
  p.h = const_cast<void*>(h);
  p.act = a;
  p.lda = lddy;
  p.ldb = F;
  p.ldc = 2 * F;
  p.R = R;
  p.S = R;
  p.N = N;
  p.K = F;
  p.m_splits = m_splits;
  p.G = G;
  p.ws = usable_workspace(workspace);
  return hip_status(mx::launch_ragged_gated_bwd(type == MXFP8_TYPE_F16, p,
                                                p.ws != nullptr ? workspace_bytes : 0, as_stream(stream)),
                    fn);
}

mxfp8_status mxfp8_quantize_int8(const void* x, int32_t type, int64_t T, int64_t K, int64_t ldx,
                                 int8_t* q, float* scale, void* stream) {
  const char* fn = "mxfp8_quantize_int8";
  if (type != MXFP8_TYPE_BF16 && type != MXFP8_TYPE_F16)
    return fail(MXFP8_ENOTSUP, "%s: type %d is not supported", fn, (int)type);
  REQUIRE(T >= 0 && T <= kI32Max && K >= 1 && K <= kI32Max,
          "%s: T = %lld must be 0 to 2^31 - 1, K = %lld 1 to 2^31 - 1", fn, (long long)T,
          (long long)K);
  REQUIRE(ldx >= K, "%s: ldx = %lld is shorter than a row", fn, (long long)ldx);
  if (T == 0) return ok();
  REQUIRE(x && q && scale, "%s: NULL pointer", fn);
  REQUIRE(aligned_to(x, 2) && aligned_to(scale, 4), "%s: a pointer is not aligned to its element",
          fn);
  return hip_status(
      mx::launch_quantize_int8(x, type == MXFP8_TYPE_F16, T, K, ldx, q, scale, as_stream(stream)),
      fn);
}

mxfp8_status mxfp8_ragged_gemm_int8(const int8_t* q, int64_t ldq, const float* scale,
                                    const int8_t* w, const float* w_scale, void* c, int64_t ldc,
                                    int32_t c_type, int64_t R, int64_t S, int64_t N, int64_t K,
                                    const int64_t* m_splits, int32_t G, const int32_t* row_index,
                                    void* workspace, size_t workspace_bytes, void* stream) {
  const char* fn = "mxfp8_ragged_gemm_int8";
  if (c_type != MXFP8_TYPE_F32 && c_type != MXFP8_TYPE_BF16 && c_type != MXFP8_TYPE_F16)
    return fail(MXFP8_ENOTSUP, "%s: output type %d is not supported", fn, (int)c_type);
  mxfp8_status st = check_ragged(fn, MXFP8_LAYOUT_NT, R, S, N, K, m_splits, G, row_index);
  if (st != MXFP8_OK) return st;
  REQUIRE(K <= 131071, "%s: K = %lld: sums of over 131071 products can pass 32 bits", fn,
          (long long)K);
  REQUIRE(ldq >= K, "%s: ldq = %lld is shorter than a row", fn, (long long)ldq);
  REQUIRE(ldc >= N, "%s: ldc = %lld is shorter than a row", fn, (long long)ldc);
  if (R == 0) return ok();
  REQUIRE(c && w && w_scale && (S == 0 || (q && scale)), "%s: NULL pointer", fn);
  REQUIRE(aligned_to(scale, 4) && aligned_to(w_scale, 4) && aligned_to(c, c_type == 0 ? 4 : 2) &&
              aligned_to(row_index, 4) && aligned_to(m_splits, 8),
          "%s: a pointer is not aligned to its element", fn);
  mx::RaggedArgs p{};
  p.a = q;
  p.b = w;
  p.c = c;
  p.lda = ldq;
  p.ldb = K;
  p.ldc = ldc;
  p.R = R;
  p.S = S;
  p.N = N;
  p.K = K;
  p.m_splits = m_splits;
  p.row_index = row_index;
  p.sa = scale;
  p.sb = w_scale;
  p.G = G;
  p.ws = usable_workspace(workspace);
  return hip_status(mx::launch_ragged_gemm_int8(
                        c_type, p, p.ws != nullptr ? workspace_bytes : 0, as_stream(stream)),
                    fn);
}

mxfp8_status mxfp8_quantize_fp8(const void* x, int32_t type, int64_t T, int64_t K, int64_t ldx, uint8_t* q,
                                float* scale, void* stream) {
  const char* fn = "mxfp8_quantize_fp8";
  if (type != MXFP8_TYPE_BF16 && type != MXFP8_TYPE_F16)
    return fail(MXFP8_ENOTSUP, "%s: type %d is not supported", fn, (int)type);
  REQUIRE(T >= 0 && T <= kI32Max && K >= 1 && K <= kI32Max,
          "%s: T = %lld must be 0 to 2^31 - 1, K = %lld 1 to 2^31 - 1", fn, (long long)T,
          (long long)K);
  REQUIRE(ldx >= K, "%s: ldx = %lld is shorter than a row", fn, (long long)ldx);
  if (T == 0) return ok();
  REQUIRE(x && q && scale, "%s: NULL pointer", fn);
  REQUIRE(aligned_to(x, 2) && aligned_to(scale, 4), "%s: a pointer is not aligned to its element",
          fn);
  return hip_status(
      mx::launch_quantize_fp8(x, type == MXFP8_TYPE_F16, T, K, ldx, q, scale, as_stream(stream)), fn);
}

mxfp8_status mxfp8_quantize_fp8_weight(const void* w, int32_t type, int64_t G, int64_t N, int64_t K,
                                       uint8_t* q, float* scale, void* stream) {
  const char* fn = "mxfp8_quantize_fp8_weight";
  if (type != MXFP8_TYPE_BF16 && type != MXFP8_TYPE_F16)
    return fail(MXFP8_ENOTSUP, "%s: type %d is not supported", fn, (int)type);
  REQUIRE(G >= 0 && G <= kI32Max && N >= 1 && N <= kI32Max && K >= 1 && K <= kI32Max,
          "%s: G = %lld must be 0 to 2^31 - 1, N = %lld and K = %lld 1 to 2^31 - 1", fn, (long long)G,
          (long long)N, (long long)K);
  const int64_t each = ((N + 127) / 128) * ((K + 127) / 128);
  REQUIRE(each <= kI32Max && G * each <= kI32Max, "%s: over 2^31 - 1 blocks", fn);
  if (G == 0) return ok();
  REQUIRE(w && q && scale, "%s: NULL pointer", fn);
  REQUIRE(aligned_to(w, 2) && aligned_to(scale, 4), "%s: a pointer is not aligned to its element",
          fn);
  return hip_status(
      mx::launch_quantize_fp8_weight(w, type == MXFP8_TYPE_F16, G, N, K, q, scale, as_stream(stream)), fn);
}

size_t mxfp8_ragged_gemm_fp8_workspace_bytes(int64_t R, int64_t S, int64_t N, int64_t K, int32_t G) {
  if (R < 0 || S < 0 || N < 1 || K < 1 || G < 1 || G > mx::kRaggedMaxGroups || R > kI32Max || S > kI32Max ||
      N > kI32Max || K > kI32Max)
    return 0;
  return mx::ragged_fp8_workspace_bytes(R, S, N, K, G);
}

namespace {

mxfp8_status ragged_gemm_fp8(const char* fn, bool fast, const uint8_t* q, int64_t ldq, const float* scale,
                             const uint8_t* w, const float* w_scale, void* c, int64_t ldc, int32_t c_type, int64_t R,
                             int64_t S, int64_t N, int64_t K, const int64_t* m_splits, int32_t G,
                             const int32_t* row_index, void* workspace, size_t workspace_bytes, void* stream) {
  if (c_type != MXFP8_TYPE_F32 && c_type != MXFP8_TYPE_BF16 && c_type != MXFP8_TYPE_F16)
    return fail(MXFP8_ENOTSUP, "%s: output type %d is not supported", fn, (int)c_type);
  mxfp8_status st = check_ragged(fn, MXFP8_LAYOUT_NT, R, S, N, K, m_splits, G, row_index);
  if (st != MXFP8_OK) return st;
  REQUIRE(ldq >= K, "%s: ldq = %lld is shorter than a row", fn, (long long)ldq);
  REQUIRE(ldc >= N, "%s: ldc = %lld is shorter than a row", fn, (long long)ldc);
  if (R == 0) return ok();
  REQUIRE(c && w && w_scale && (S == 0 || (q && scale)), "%s: NULL pointer", fn);
  REQUIRE(aligned_to(scale, 4) && aligned_to(w_scale, 4) && aligned_to(c, c_type == 0 ? 4 : 2) &&
              aligned_to(row_index, 4) && aligned_to(m_splits, 8),
          "%s: a pointer is not aligned to its element", fn);
  mx::RaggedArgs p{};
  p.a = q;
  p.b = w;
  p.c = c;
  p.lda = ldq;
  p.ldb = K;
  p.ldc = ldc;
  p.R = R;
  p.S = S;
  p.N = N;
  p.K = K;
  p.m_splits = m_splits;
  p.row_index = row_index;
  p.sa = scale;
  p.sb = w_scale;
  p.G = G;
  p.ws = usable_workspace(workspace);
  return hip_status(mx::launch_ragged_gemm_fp8(
                        c_type, fast, p, p.ws != nullptr ? workspace_bytes : 0, as_stream(stream)),
                    fn);
}

}  // namespace

mxfp8_status mxfp8_ragged_gemm_fp8(const uint8_t* q, int64_t ldq, const float* scale, const uint8_t* w,
                                   const float* w_scale, void* c, int64_t ldc, int32_t c_type, int64_t R,
                                   int64_t S, int64_t N, int64_t K, const int64_t* m_splits, int32_t G,
                                   const int32_t* row_index, void* workspace, size_t workspace_bytes,
                                   void* stream) {
  return ragged_gemm_fp8("mxfp8_ragged_gemm_fp8", false, q, ldq, scale, w, w_scale, c, ldc, c_type, R, S, N, K,
                         m_splits, G, row_index, workspace, workspace_bytes, stream);
}

mxfp8_status mxfp8_ragged_gemm_fp8_fast(const uint8_t* q, int64_t ldq, const float* scale, const uint8_t* w,
                                        const float* w_scale, void* c, int64_t ldc, int32_t c_type, int64_t R,
                                        int64_t S, int64_t N, int64_t K, const int64_t* m_splits, int32_t G,
                                        const int32_t* row_index, void* workspace, size_t workspace_bytes,
                                        void* stream) {
  const char* fn = "mxfp8_ragged_gemm_fp8_fast";
  if (c_type == MXFP8_TYPE_F32) return fail(MXFP8_ENOTSUP, "%s: fp32 results need fp32 sums", fn);
  return ragged_gemm_fp8(fn, true, q, ldq, scale, w, w_scale, c, ldc, c_type, R, S, N, K, m_splits, G, row_index,
                         workspace, workspace_bytes, stream);
}

namespace {

constexpr int32_t kRouteMaxExperts = 1024;

mxfp8_status check_route(const char* fn, int32_t type, int64_t T, int32_t E, int32_t top_k) {
  if (type != MXFP8_TYPE_F32 && type != MXFP8_TYPE_BF16 && type != MXFP8_TYPE_F16)
    return fail(MXFP8_ENOTSUP, "%s: logits type %d is not supported", fn, (int)type);
  REQUIRE(E >= 1 && E <= kRouteMaxExperts, "%s: E = %d must be 1 to %d", fn, (int)E,
          kRouteMaxExperts);
  REQUIRE(top_k >= 1 && top_k <= 16 && top_k <= E, "%s: top_k = %d must be 1 to min(E, 16)", fn,
          (int)top_k);
  REQUIRE(T >= 0 && T <= kI32Max / top_k, "%s: T = %lld: T * top_k must be below 2^31", fn,
          (long long)T);
  return MXFP8_OK;
}

mxfp8_status check_join(const char* fn, int32_t type, int64_t T, int64_t R, int64_t H,
                        int32_t top_k) {
  if (type != MXFP8_TYPE_BF16 && type != MXFP8_TYPE_F16)
    return fail(MXFP8_ENOTSUP, "%s: type %d is not supported", fn, (int)type);
  REQUIRE(T >= 0 && R >= 0 && T <= kI32Max && R <= kI32Max,
          "%s: T = %lld and R = %lld must be 0 to 2^31 - 1", fn, (long long)T, (long long)R);
  REQUIRE(H >= 1 && H <= kI32Max, "%s: H = %lld must be 1 to 2^31 - 1", fn, (long long)H);
  REQUIRE(top_k >= 1 && top_k <= 16, "%s: top_k = %d must be 1 to 16", fn, (int)top_k);
  return MXFP8_OK;
}

}  // namespace

size_t mxfp8_moe_route_workspace_bytes(int64_t T, int32_t E) {
  if (T < 0 || T > kI32Max || E < 1 || E > kRouteMaxExperts) return 0;
  return mx::route_workspace_bytes(T, E);
}

mxfp8_status mxfp8_moe_route(const void* logits, int32_t type, int64_t T, int32_t E,
                             int32_t top_k, int32_t renormalize, const uint8_t* token_mask,
                             int32_t* ids, float* weights, int64_t* m_splits, int32_t* row_token,
                             int32_t* row_pos, void* workspace, size_t workspace_bytes,
                             void* stream) {
  const char* fn = "mxfp8_moe_route";
  mxfp8_status st = check_route(fn, type, T, E, top_k);
  if (st != MXFP8_OK) return st;
  REQUIRE(m_splits != nullptr, "%s: m_splits is NULL", fn);
  REQUIRE(T == 0 || (logits && ids && weights && row_token && row_pos), "%s: NULL pointer", fn);
  const size_t need = mx::route_workspace_bytes(T, E);
  REQUIRE(need == 0 || (workspace != nullptr && workspace_bytes >= need),
          "%s: needs a workspace of %zu bytes", fn, need);
  REQUIRE(aligned_to(logits, type == 0 ? 4 : 2) && aligned_to(ids, 4) && aligned_to(weights, 4) &&
              aligned_to(m_splits, 8) && aligned_to(row_token, 4) && aligned_to(row_pos, 4) &&
              (need == 0 || aligned_to(workspace, 4)),
          "%s: a pointer is not aligned to its element", fn);
  return hip_status(mx::launch_route(logits, type, T, E, top_k, renormalize != 0, token_mask, ids,
                                     weights, m_splits, row_token, row_pos, workspace,
                                     as_stream(stream)),
                    fn);
}

mxfp8_status mxfp8_moe_route_bwd(const void* logits, int32_t type, int64_t T, int32_t E,
                                 int32_t top_k, int32_t renormalize, const int32_t* ids,
                                 const float* weights, const float* dweights, void* dlogits,
                                 void* stream) {
  const char* fn = "mxfp8_moe_route_bwd";
  mxfp8_status st = check_route(fn, type, T, E, top_k);
  if (st != MXFP8_OK) return st;
  if (T == 0) return ok();
  REQUIRE(logits && ids && weights && dweights && dlogits, "%s: NULL pointer", fn);
  REQUIRE(aligned_to(logits, type == 0 ? 4 : 2) && aligned_to(dlogits, type == 0 ? 4 : 2) &&
              aligned_to(ids, 4) && aligned_to(weights, 4) && aligned_to(dweights, 4),
          "%s: a pointer is not aligned to its element", fn);
  return hip_status(mx::launch_route_bwd(logits, type, T, E, top_k, renormalize != 0, ids, weights,
                                         dweights, dlogits, as_stream(stream)),
                    fn);
}

mxfp8_status mxfp8_moe_combine(const void* y, int32_t type, int64_t T, int64_t R, int64_t H,
                               int32_t top_k, const int32_t* row_pos, const float* weights,
                               void* out, void* stream) {
  const char* fn = "mxfp8_moe_combine";
  mxfp8_status st = check_join(fn, type, T, R, H, top_k);
  if (st != MXFP8_OK) return st;
  if (T == 0) return ok();
  REQUIRE(row_pos && out && (y || R == 0), "%s: NULL pointer", fn);
  REQUIRE(aligned_to(y, 2) && aligned_to(out, 2) && aligned_to(row_pos, 4) &&
              aligned_to(weights, 4),
          "%s: a pointer is not aligned to its element", fn);
  return hip_status(mx::launch_join(y, type == MXFP8_TYPE_F16, T, R, H, top_k, row_pos, weights,
                                    out, as_stream(stream)),
                    fn);
}

mxfp8_status mxfp8_moe_combine_bwd(const void* dout, const void* y, int32_t type, int64_t T,
                                   int64_t R, int64_t H, int32_t top_k, const int32_t* row_pos,
                                   const float* weights, void* dy, float* dweights,
                                   void* stream) {
  const char* fn = "mxfp8_moe_combine_bwd";
  mxfp8_status st = check_join(fn, type, T, R, H, top_k);
  if (st != MXFP8_OK) return st;
  REQUIRE(dy != nullptr || dweights != nullptr || R == 0 || T == 0, "%s: no output asked for", fn);
  if (T == 0 || (dy == nullptr && dweights == nullptr)) return ok();
  REQUIRE(dout && row_pos && (dweights == nullptr || y || R == 0), "%s: NULL pointer", fn);
  REQUIRE(aligned_to(dout, 2) && aligned_to(y, 2) && aligned_to(dy, 2) && aligned_to(row_pos, 4) &&
              aligned_to(weights, 4) && aligned_to(dweights, 4),
          "%s: a pointer is not aligned to its element", fn);
  return hip_status(mx::launch_join_bwd(dout, y, type == MXFP8_TYPE_F16, T, R, H, top_k, row_pos,
                                        weights, dy, dweights, as_stream(stream)),
                    fn);
}

namespace {

mxfp8_status check_norm(const char* fn, int32_t x_type, int32_t type, int32_t w_type, int64_t T, int64_t H,
                        float eps, const void* f, const float* gate, const void* post, const void* pre) {
  if (type != MXFP8_TYPE_BF16 && type != MXFP8_TYPE_F16)
    return fail(MXFP8_ENOTSUP, "%s: type %d is not supported", fn, (int)type);
  if (x_type != MXFP8_TYPE_F32 && x_type != type)
    return fail(MXFP8_ENOTSUP, "%s: residual type %d is not supported", fn, (int)x_type);
  if (w_type != MXFP8_TYPE_F32 && w_type != type)
    return fail(MXFP8_ENOTSUP, "%s: weight type %d is not supported", fn, (int)w_type);
  REQUIRE(T >= 0 && T <= kI32Max, "%s: T = %lld must be 0 to 2^31 - 1", fn, (long long)T);
  REQUIRE(H >= 1 && H <= mx::norm_max_hidden(), "%s: H = %lld must be 1 to %lld", fn, (long long)H,
          (long long)mx::norm_max_hidden());
  REQUIRE(eps >= 0.f && eps <= 3.4028235e38f, "%s: eps must be a finite number from 0 up", fn);
  REQUIRE(f != nullptr || T == 0 || (gate == nullptr && post == nullptr), "%s: gate and post_weight need f", fn);
  const size_t w = w_type == MXFP8_TYPE_F32 ? 4 : 2;
  REQUIRE(aligned_to(f, 2) && aligned_to(gate, 4) && aligned_to(post, w) && aligned_to(pre, w),
          "%s: a pointer is not aligned to its element", fn);
  return MXFP8_OK;
}

}  // namespace

mxfp8_status mxfp8_residual_norm(const void* x, int32_t x_type, const void* f, int32_t type, int64_t T,
                                 int64_t H, float residual_scale, const float* gate,
                                 const void* post_weight, const void* pre_weight, int32_t w_type, float eps,
                                 void* r, void* y, void* stream) {
  const char* fn = "mxfp8_residual_norm";
  mxfp8_status st = check_norm(fn, x_type, type, w_type, T, H, eps, f, gate, post_weight, pre_weight);
  if (st != MXFP8_OK) return st;
  if (T == 0) return ok();
  REQUIRE(x != nullptr, "%s: x is NULL", fn);
  REQUIRE((f != nullptr) == (r != nullptr), "%s: r goes with f", fn);
  REQUIRE((pre_weight != nullptr) == (y != nullptr), "%s: y goes with pre_weight", fn);
  REQUIRE(r != nullptr || y != nullptr, "%s: no output asked for", fn);
  const size_t xs = x_type == MXFP8_TYPE_F32 ? 4 : 2;
  REQUIRE(aligned_to(x, xs) && aligned_to(r, xs) && aligned_to(y, 2),
          "%s: a pointer is not aligned to its element", fn);
  return hip_status(mx::launch_residual_norm(x, x_type == MXFP8_TYPE_F32, f, type == MXFP8_TYPE_F16, T, H,
                                             residual_scale, gate, post_weight, pre_weight,
                                             w_type == MXFP8_TYPE_F32, eps, r, y, as_stream(stream)),
                    fn);
}

size_t mxfp8_residual_norm_bwd_workspace_bytes(int64_t T, int64_t H) {
  if (T < 0 || T > kI32Max || H < 1 || H > mx::norm_max_hidden()) return 0;
  return mx::norm_bwd_workspace_bytes(T, H);
}

mxfp8_status mxfp8_residual_norm_bwd(const void* dy, const void* dr, const void* r, int32_t x_type,
                                     const void* f, int32_t type, int64_t T, int64_t H,
                                     float residual_scale, const float* gate, const void* post_weight,
                                     const void* pre_weight, int32_t w_type, float eps, void* dx, void* df,
                                     float* dgate, float* dpost_weight, float* dpre_weight,
                                     void* workspace, size_t workspace_bytes, void* stream) {
  const char* fn = "mxfp8_residual_norm_bwd";
  mxfp8_status st = check_norm(fn, x_type, type, w_type, T, H, eps, f, gate, post_weight, pre_weight);
  if (st != MXFP8_OK) return st;
  REQUIRE(T == 0 || dx || df || dgate || dpost_weight || dpre_weight, "%s: no output asked for", fn);
  REQUIRE(dpost_weight == nullptr || post_weight != nullptr, "%s: dpost_weight needs post_weight", fn);
  REQUIRE(dpre_weight == nullptr || pre_weight != nullptr, "%s: dpre_weight needs pre_weight", fn);
  REQUIRE(dgate == nullptr || gate != nullptr, "%s: dgate needs gate", fn);
  const size_t need = dpost_weight != nullptr || dpre_weight != nullptr ? mx::norm_bwd_workspace_bytes(T, H) : 0;
  REQUIRE(need == 0 || (workspace != nullptr && workspace_bytes >= need && aligned_to(workspace, 4)),
          "%s: needs a workspace of %zu bytes", fn, need);
  if (T > 0) {
    REQUIRE(dy != nullptr || dr != nullptr, "%s: neither dy nor dr", fn);
    REQUIRE(dy == nullptr || pre_weight != nullptr, "%s: dy goes with pre_weight", fn);
    REQUIRE(dpre_weight == nullptr || dy != nullptr, "%s: dpre_weight needs dy", fn);
    REQUIRE(dy == nullptr || r != nullptr, "%s: r is NULL", fn);
    REQUIRE(f != nullptr || df == nullptr, "%s: df needs f", fn);
  }
  const size_t xs = x_type == MXFP8_TYPE_F32 ? 4 : 2;
  REQUIRE(aligned_to(dy, 2) && aligned_to(dr, xs) && aligned_to(r, xs) && aligned_to(dx, xs) &&
              aligned_to(df, 2) && aligned_to(dgate, 4) && aligned_to(dpost_weight, 4) &&
              aligned_to(dpre_weight, 4),
          "%s: a pointer is not aligned to its element", fn);
  return hip_status(
      mx::launch_residual_norm_bwd(dy, dr, r, x_type == MXFP8_TYPE_F32, f, type == MXFP8_TYPE_F16, T, H,
                                   f != nullptr ? residual_scale : 1.f, gate, post_weight, pre_weight,
                                   w_type == MXFP8_TYPE_F32, eps, dx, df, dgate, dpost_weight, dpre_weight,
                                   workspace, as_stream(stream)),
      fn);
}

}  // extern "C"
