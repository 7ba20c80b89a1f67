// What the operators beside the optimizer step share on the host: the
// per-device facts that every call needs, and the check of the error word.
#include "op_common.cuh"

namespace ma {
namespace {

__device__ int g_op_error;  // first error code of a bounded wait that ran out

struct DeviceFacts {
  std::atomic<bool> ready;
  int sms;
  int* err;
};
DeviceFacts g_facts[kOpMaxDevices];

cudaError_t look_up(int dev, int* sms, int** err) {
  void* p = nullptr;
  cudaError_t e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess) e = cudaGetSymbolAddress(&p, g_op_error);
  *err = static_cast<int*>(p);
  return e;
}

}  // namespace

cudaError_t op_device(int* sms, int** err) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  // A thread that has made no CUDA call yet (one of autograd's, say) has no
  // current context, without which the driver encodes no tensor map.
  thread_local int bound = -1;
  if (bound != dev) {
    e = cudaSetDevice(dev);
    if (e != cudaSuccess) return e;
    bound = dev;
  }
  if (dev < 0 || dev >= kOpMaxDevices) return look_up(dev, sms, err);
  DeviceFacts& f = g_facts[dev];
  if (!f.ready.load(std::memory_order_acquire)) {
    // racing threads write the same values
    e = look_up(dev, sms, err);
    if (e != cudaSuccess) return e;
    f.sms = *sms;
    f.err = *err;
    f.ready.store(true, std::memory_order_release);
  }
  *sms = f.sms;
  *err = f.err;
  return cudaSuccess;
}

}  // namespace ma

using namespace ma;

extern "C" MA_API ma_status muon_adamw_operators_check(void* cuda_stream) {
  int sms = 0, *p = nullptr, code = 0;
  const cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  cudaError_t e = op_device(&sms, &p);
  if (e == cudaSuccess) e = cudaMemcpyAsync(&code, p, sizeof code, cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e == cudaSuccess && code != 0) {
    e = cudaMemsetAsync(p, 0, sizeof code, s);
    if (e == cudaSuccess)
      return op_fail(MA_ERR_DEVICE_CHECK, "a kernel's bounded wait ran out (code 0x%x); its results are not valid", code);
  }
  if (e != cudaSuccess) return op_cuda(e, "operators check");
  clear_last_error();
  return MA_OK;
}
