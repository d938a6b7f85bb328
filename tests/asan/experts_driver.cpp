// Host-side sanitizer check of the entry points of gemm_experts.h, and a view of their kernel choice (no
// GPU needed): xapi.cpp is compiled into this program with launchers that only print what they are asked
// to launch, and the calls named on standard input are made with a handle of 256 compute units and
// addresses that nothing dereferences.
//
// A line of input, one of
//   mx kernel groups M N K lda ldb ldc ldsa ldsb stride skew c_type epilogue   (-1: the dense one)
//   moves T top K ld rows type          dispatch, combine, its gradient and quantization with places
//   route T E top groups top_groups ldl type score renorm               and its gradient
// skew: bytes that A starts after a multiple of 16.  A line of output: the statuses and launches.
#include "xapi.cpp"

#include <stdio.h>
#include <string.h>

#include <string>

namespace {
std::string launched;
hipError_t note(const char* what, int a = -1, int b = -1) {
  char s[100];
  snprintf(s, sizeof s, a < 0 ? " %s" : b < 0 ? " %s %d" : " %s %d %d", what, a, b);
  launched += s;
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
hipError_t launch_route(const RouteArgs&, hipStream_t) { return note("route"); }
hipError_t launch_route_grad(const RouteGradArgs&, hipStream_t) { return note("grad"); }
hipError_t launch_dispatch_rows(const RowArgs&, int, hipStream_t) { return note("dispatch"); }
hipError_t launch_combine_rows(const RowArgs&, int, hipStream_t) { return note("combine"); }
hipError_t launch_combine_rows_grad(const RowGradArgs&, int, hipStream_t) { return note("grad"); }
hipError_t launch_quantize_mx(const QuantizeMxArgs&, int, hipStream_t) { return note("quantize"); }
hipError_t launch_stream_mx(const GemmParams&, const GroupArgs&, int, int r, int c, hipStream_t) { return note("stream", r, c); }
hipError_t launch_grouped_mx_f16(const GemmParams&, const GroupArgs&, int t, int, hipStream_t) { return note("tile", t); }
hipError_t launch_grouped_mx_bf16(const GemmParams&, const GroupArgs&, int t, int, hipStream_t) { return note("tile", t); }
hipError_t launch_grouped_mx_f32(const GemmParams&, const GroupArgs&, int t, int, hipStream_t) { return note("tile", t); }
}  // namespace tgemm

int main() {
  gemm_handle h{};
  h.magic = tgemm::kHandleMagic;
  h.cu_count = 256;
  // 2^59 bytes apart
  auto far = [](int i) { return at((int64_t)i << 59); };
  char call[32];
  while (scanf("%31s", call) == 1) {
    launched.clear();
    if (!strcmp(call, "mx")) {
      long long G, M, N, K, lda, ldb, ldc, ldsa, ldsb, stride;
      int kernel, skew, ct, epi;
      if (scanf("%d %lld %lld %lld %lld %lld %lld %lld %lld %lld %lld %d %d %d", &kernel, &G, &M, &N, &K, &lda, &ldb, &ldc,
                &ldsa, &ldsb, &stride, &skew, &ct, &epi) != 14)
        return 1;
      const long long blocks = (K / 32 + 15) / 16 * 16;
      if (lda < 0) lda = K;
      if (ldb < 0) ldb = K;
      if (ldc < 0) ldc = N;
      if (ldsa < 0) ldsa = blocks;
      if (ldsb < 0) ldsb = blocks;
      if (stride < 0) stride = N * ldb;
      const gemm_status_t st = gemm_run_grouped_mx(
          &h, (gemm_grouped_kernel_t)kernel, nullptr, G, (const int64_t*)far(1), M, N, K, 1.f, (uint8_t*)far(2) + skew, lda,
          (uint8_t*)far(3), ldsa, far(4), ldb, stride, (uint8_t*)far(5), ldsb, N * ldsb, 0.f, far(6), ldc, GEMM_E2M1,
          (gemm_dtype_t)ct, (uint32_t)epi, nullptr);
      printf("%d%s\n", (int)st, launched.c_str());
    } else if (!strcmp(call, "moves")) {
      long long T, top, K, ld, R;
      int t;
      if (scanf("%lld %lld %lld %lld %lld %d", &T, &top, &K, &ld, &R, &t) != 6) return 1;
      const gemm_dtype_t type = (gemm_dtype_t)t;
      int32_t* const place = (int32_t*)far(1);
      float* const w = (float*)far(2);
      const int a = gemm_dispatch_rows(&h, nullptr, T, top, K, far(3), ld, type, place, R, far(5), ld);
      const int b = gemm_combine_rows(&h, nullptr, T, top, K, far(5), ld, type, place, R, w, 0.f, far(3), ld);
      const int c = gemm_combine_rows_grad(&h, nullptr, T, top, K, far(3), ld, far(5), ld, type, place, R, w, far(7), ld,
                                           (float*)far(9));
      const int d = gemm_quantize_mx(&h, nullptr, T, K, far(3), ld, type, top, place, R, far(5), ld, GEMM_E2M1,
                                     (uint8_t*)far(7), ld);
      printf("%d %d %d %d%s\n", a, b, c, d, launched.c_str());
    } else {
      long long T, E, top, groups, best, ldl;
      int type, score, renorm;
      if (scanf("%lld %lld %lld %lld %lld %lld %d %d %d", &T, &E, &top, &groups, &best, &ldl, &type, &score, &renorm) != 9)
        return 1;
      const int64_t need = gemm_route_workspace_bytes(T, E);
      const int a = gemm_route(&h, nullptr, T, E, top, far(1), ldl, (gemm_dtype_t)type, (gemm_score_t)score, (float*)far(2),
                               groups, best, 1, renorm, 1.f, (int32_t*)far(3), (float*)far(4), (int32_t*)far(5),
                               (int64_t*)far(6), far(7), need < 0 ? 0 : need);
      const int b = gemm_route_grad(&h, nullptr, T, E, top, far(1), ldl, (gemm_dtype_t)type, (gemm_score_t)score, renorm, 1.f,
                                    (int32_t*)far(3), (float*)far(4), far(8), ldl);
      printf("%lld %d %d%s\n", (long long)need, a, b, launched.c_str());
    }
  }
  return 0;
}
