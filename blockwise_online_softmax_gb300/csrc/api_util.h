// Helpers shared by the host units of the C ABI (ra_api.cu, serve_api.cu):
// errors, argument checks, tracing, the scratch pool and the tensor-map
// encoder.  They are defined in ra_api.cu.
#pragma once
#include <initializer_list>

#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

namespace ra {
namespace api {

// Default wait bound for the kernels' mbarrier waits: 2^31 SM cycles,
// about one second at the maximum SM clock.
constexpr long long kWaitLimit = 1LL << 31;

// Sets the calling thread's message and returns `status`.
int fail(int status, const char* fmt, ...);
int cuda_fail(cudaError_t e, const char* what);
bool aligned16(const void* p);

// Brackets one kernel launch with an event pair on its stream while
// tracing is on.
struct TraceScope {
  int kind;
  cudaStream_t st;
  cudaEvent_t a = nullptr, b = nullptr;
  bool on = false;
  TraceScope(int k, cudaStream_t s);
  void done(bool launched);
};

// Stream-ordered allocation from the current device's pool; the buffer is
// returned with cudaFreeAsync like any other.
cudaError_t scratch_alloc(void** p, size_t bytes, cudaStream_t st);

// Looks cuTensorMapEncodeTiled up once; encode_tiled may be called when it is RA_OK.
int get_encoder();
// cuTensorMapEncodeTiled, which wants a current context.  A thread that has made no
// call of the runtime with work for the device yet has none: there it is made current.
CUresult encode_tiled(CUtensorMap* map, CUtensorMapDataType type, cuuint32_t rank, void* base, const cuuint64_t* dims,
                      const cuuint64_t* strides, const cuuint32_t* box, const cuuint32_t* estr,
                      CUtensorMapInterleave interleave, CUtensorMapSwizzle swizzle, CUtensorMapL2promotion promotion,
                      CUtensorMapFloatOOBfill fill);

int check_common(int d, int heads, int dtype);
int check_heads(int heads, int kv_heads);
// Every pointer given, and 16-byte aligned.
int check_ptrs(std::initializer_list<const void*> ps);

}  // namespace api
}  // namespace ra
