// Graphs under capture and their end (declared in include/pagedkv.h). The watch is a user object
// of the captured graph: CUDA holds it for the graph and for its executables and calls
// ended() from a thread of its own when the last of them goes.
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>
#include <new>

#include "pagedkv.h"

namespace {

struct Watch {
  std::atomic<int> gone{0};
};

void CUDART_CB ended(void* watch) { static_cast<Watch*>(watch)->gone.store(1, std::memory_order_release); }

int failed() {
  cudaGetLastError();
  return PKV_ERR_CUDA;
}

}  // namespace

extern "C" {

int pkv_capture_watch(void* stream, uint64_t* id, void** watch) {
  if (!id) return PKV_ERR_INVALID_ARGUMENT;
  *id = 0;
  if (watch) *watch = nullptr;
  cudaStreamCaptureStatus status = cudaStreamCaptureStatusNone;
  unsigned long long capture = 0;
  cudaGraph_t graph = nullptr;
  if (cudaStreamGetCaptureInfo(static_cast<cudaStream_t>(stream), &status, &capture, &graph, nullptr, nullptr, nullptr) !=
          cudaSuccess ||
      status == cudaStreamCaptureStatusInvalidated)
    return failed();
  if (status == cudaStreamCaptureStatusNone) return PKV_OK;
  if (watch) {
    Watch* w = new (std::nothrow) Watch;
    if (!w) return PKV_ERR_CUDA;
    cudaUserObject_t object = nullptr;
    if (cudaUserObjectCreate(&object, w, ended, 1, cudaUserObjectNoDestructorSync) != cudaSuccess) {
      delete w;
      return failed();
    }
    if (cudaGraphRetainUserObject(graph, object, 1, cudaGraphUserObjectMove) != cudaSuccess) {
      cudaUserObjectRelease(object, 1);   // (calls ended() later: its word stays)
      return failed();
    }
    *watch = w;
  }
  *id = capture;
  return PKV_OK;
}

int pkv_capture_gone(void* watch) {
  Watch* w = static_cast<Watch*>(watch);
  if (!w || w->gone.load(std::memory_order_acquire) == 0) return 0;
  delete w;
  return 1;
}

}  // extern "C"
