/* launch_recorder.c -- stands in for the HIP runtime's launch, so that the library's choice of kernel shows on a
 * machine without a GPU (launches.py).  Loaded with its symbols global before the library, whose references
 * then bind here: kernels are registered under their names, the current device is number 0, and a launch is
 * recorded and not made. */
#define __HIP_PLATFORM_AMD__
#include <hip/hip_runtime_api.h>

#include <stddef.h>
#include <string.h>

enum { KERNELS = 4096 };
static struct {
  const void *host;
  const char *name;
} kernels[KERNELS];
static int count;
static struct {
  const char *name;
  unsigned grid, block;
} last;

void **__hipRegisterFatBinary(const void *data) {
  static void *modules;
  (void)data;
  return &modules;
}
void __hipUnregisterFatBinary(void **modules) { (void)modules; }
void __hipRegisterFunction(void **modules, const void *host, char *device, const char *name, unsigned threads, void *tid,
                           void *bid, void *block, void *grid, int *size) {
  (void)modules, (void)device, (void)threads, (void)tid, (void)bid, (void)block, (void)grid, (void)size;
  if (count < KERNELS) kernels[count].host = host, kernels[count++].name = name;
}
hipError_t hipGetDevice(int *device) {
  *device = 0;
  return hipSuccess;
}
hipError_t hipLaunchKernel(const void *host, dim3 grid, dim3 block, void **args, size_t shared, hipStream_t stream) {
  (void)args, (void)shared, (void)stream;
  last.name = NULL;
  for (int i = 0; i < count; i++)
    if (kernels[i].host == host) last.name = kernels[i].name;
  last.grid = grid.x, last.block = block.x;
  return last.name && grid.y == 1 && grid.z == 1 && block.y == 1 && block.z == 1 ? hipSuccess : hipErrorInvalidDeviceFunction;
}

const char *recorded_kernel(void) { return last.name; }
unsigned recorded_grid(void) { return last.grid; }
unsigned recorded_block(void) { return last.block; }
