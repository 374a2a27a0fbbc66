// Waits of csrc/tc.cuh with a limit of eight tries (16 us), on a barrier that nobody arrives at or
// that has been arrived at; compiled and called by test_wait_limit.py.
#include "../sparse_memory_linear_b200/csrc/tc.cuh"

using namespace sdm;

__global__ void __launch_bounds__(128) wait_kernel(int arrive, int* out) {
  __shared__ __align__(8) unsigned long long barrier;
  __shared__ uint32_t tmem;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t bar = smem_addr(&barrier);
  if (warp == 0) tmem_alloc(smem_addr(&tmem), 32);
  if (threadIdx.x == 0) {
    mbar_init(bar, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (arrive && threadIdx.x == 0) mbar_arrive(bar);
  __syncwarp();
  bool ok = true;
  if (warp < 3) {
    ok = mbar_wait_warp<8>(bar, 0);
  } else {  // one lane on its own, as the loads' warps wait
    if (lane == 0) ok = mbar_wait<8>(bar, 0);
    ok = __shfl_sync(FULL_MASK, (int)ok, 0);
  }
  const int elected = elect_one();  // a whole warp gets here
  out[threadIdx.x] = (ok ? 1 : 0) | elected << 1;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tmem_free(tmem, 32);
  if (!ok) record_status(STATUS_TIMEOUT);
}

// out: 128 ints on the host; *status: the status word, read and cleared.  Returns a cudaError.
extern "C" int run_wait(int arrive, int* out, unsigned* status) {
  int* dev = nullptr;
  cudaError_t e = cudaMalloc(&dev, 128 * sizeof(int));
  if (e != cudaSuccess) return e;
  wait_kernel<<<1, 128>>>(arrive, dev);
  e = cudaGetLastError();
  if (e == cudaSuccess) e = cudaMemcpy(out, dev, 128 * sizeof(int), cudaMemcpyDeviceToHost);
  if (e == cudaSuccess) e = cudaMemcpyFromSymbol(status, g_status, sizeof(unsigned));
  const unsigned none = 0;
  if (e == cudaSuccess) e = cudaMemcpyToSymbol(g_status, &none, sizeof(unsigned));
  const cudaError_t f = cudaFree(dev);
  return e != cudaSuccess ? e : f;
}
