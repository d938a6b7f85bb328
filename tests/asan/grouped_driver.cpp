// Host-side sanitizer check of the grouped and 8-bit integer entry points, and a view of their kernel
// choice (no GPU needed): gapi.cpp is compiled into this program with launchers that only print what
// they are asked to launch, and the calls named on standard input are made with a handle of 256
// compute units and addresses that nothing dereferences.
//
// A line of input: call kernel groups M N K transB lda ldb ldc stride skew type c_type dbias
//   call: grouped, wgrad, i8 or grouped_i8; stride: B's, or for wgrad C's; skew: bytes that A starts
//   after a multiple of 16; lda, ldb, ldc or stride of -1: the dense one.
// A line of output: the status, and the launch ("none" without one).
#include "gapi.cpp"

#include <stdio.h>
#include <string.h>

#include <string>

namespace {
char launched[200];
hipError_t note(const char* what, const tgemm::GemmParams& p, int a, int b) {
  snprintf(launched, sizeof launched, "%s %d %d (%d x %d x %d)", what, a, b, p.M, p.N, p.K);
  return hipSuccess;
}
void* at(int64_t n) { return reinterpret_cast<void*>(n); }
}  // namespace

extern "C" hipError_t hipGetDevice(int* d) {
  *d = 0;
  return hipSuccess;
}
extern "C" hipError_t hipSetDevice(int) { return hipSuccess; }

namespace tgemm {
hipError_t launch_grouped_f16(const GemmParams& p, const GroupArgs&, bool, int t, int, hipStream_t) { return note("tile", p, t, 0); }
hipError_t launch_grouped_bf16(const GemmParams& p, const GroupArgs&, bool, int t, int, hipStream_t) { return note("tile", p, t, 0); }
hipError_t launch_grouped_i8_f16(const GemmParams& p, const GroupArgs&, bool, int t, int, hipStream_t) { return note("tile", p, t, 0); }
hipError_t launch_grouped_i8_bf16(const GemmParams& p, const GroupArgs&, bool, int t, int, hipStream_t) { return note("tile", p, t, 0); }
hipError_t launch_grouped_i8_f32(const GemmParams& p, const GroupArgs&, bool, int t, int, hipStream_t) { return note("tile", p, t, 0); }
hipError_t launch_grouped_wgrad_f16(const GemmParams& p, const GroupArgs&, const BiasGrad&, int, int t, hipStream_t) { return note("tile", p, t, 0); }
hipError_t launch_grouped_wgrad_bf16(const GemmParams& p, const GroupArgs&, const BiasGrad&, int, int t, hipStream_t) { return note("tile", p, t, 0); }
hipError_t launch_stream_f16(const GemmParams& p, const GroupArgs&, int, bool, int rows, int waves, hipStream_t) { return note("stream", p, rows, waves); }
hipError_t launch_stream_bf16(const GemmParams& p, const GroupArgs&, int, bool, int rows, int waves, hipStream_t) { return note("stream", p, rows, waves); }
hipError_t launch_stream_i8(const GemmParams& p, const GroupArgs&, int, bool, int rows, int waves, hipStream_t) { return note("stream", p, rows, waves); }
hipError_t launch_quantize_rows(const void*, int64_t, int, int, int, int8_t*, int64_t, float*, hipStream_t) { return hipSuccess; }
}  // namespace tgemm

int main() {
  gemm_handle h{};
  h.magic = tgemm::kHandleMagic;
  h.cu_count = 256;
  char call[32];
  int kernel, tb, skew, type, ct, bias;
  long long G, M, N, K, lda, ldb, ldc, stride;
  while (scanf("%31s %d %lld %lld %lld %lld %d %lld %lld %lld %lld %d %d %d %d", call, &kernel, &G, &M, &N, &K, &tb, &lda,
               &ldb, &ldc, &stride, &skew, &type, &ct, &bias) == 15) {
    // 2^60 bytes apart
    const int64_t* const off = static_cast<int64_t*>(at(1ll << 60));
    void* const A = at((2ll << 60) + skew);
    void* const B = at(3ll << 60);
    void* const C = at(4ll << 60);
    float* const sa = static_cast<float*>(at(5ll << 60));
    float* const sb = static_cast<float*>(at(6ll << 60));
    float* const db = bias ? static_cast<float*>(at((6ll << 60) + (1ll << 59))) : nullptr;
    const gemm_grouped_kernel_t k = static_cast<gemm_grouped_kernel_t>(kernel);
    const bool w = !strcmp(call, "wgrad");
    if (lda < 0) lda = K;
    if (w) {
      if (ldb < 0) ldb = N;
      if (ldc < 0) ldc = tb ? K : N;
      if (stride < 0) stride = (tb ? N : K) * ldc;
    } else {
      if (ldb < 0) ldb = tb ? K : N;
      if (ldc < 0) ldc = N;
      if (stride < 0) stride = (tb ? N : K) * ldb;
    }
    strcpy(launched, "none");
    gemm_status_t st;
    if (w)
      st = gemm_run_grouped_wgrad(&h, k, nullptr, G, off, M, N, K, tb, 1.f, A, lda, B, ldb, 0.f, C, ldc, stride,
                                  (gemm_dtype_t)type, (gemm_dtype_t)ct, db);
    else if (!strcmp(call, "grouped"))
      st = gemm_run_grouped(&h, k, nullptr, G, off, M, N, K, tb, 1.f, A, lda, B, ldb, stride, 0.f, C, ldc,
                            (gemm_dtype_t)type, 0, nullptr);
    else if (!strcmp(call, "i8"))
      st = gemm_run_i8(&h, k, nullptr, M, N, K, tb, 1.f, static_cast<int8_t*>(A), lda, sa, static_cast<int8_t*>(B), ldb,
                       sb, 0.f, C, ldc, (gemm_dtype_t)ct, 0, nullptr);
    else
      st = gemm_run_grouped_i8(&h, k, nullptr, G, off, M, N, K, tb, 1.f, static_cast<int8_t*>(A), lda, sa,
                               static_cast<int8_t*>(B), ldb, stride, sb, 0.f, C, ldc, (gemm_dtype_t)ct, 0, nullptr);
    printf("%d %s\n", (int)st, launched);
  }
  return 0;
}
