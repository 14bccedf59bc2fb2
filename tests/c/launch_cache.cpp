// csrc/launch.cuh with a stand-in for the runtime: a kernel's limit of shared
// memory is raised once a device and thread, however many kernels there are.
#include <cuda_runtime.h>

#include <cstdio>
#include <cstdlib>
#include <thread>

#include "launch.cuh"

static int device = 0, fail = 0;
static thread_local int raised = 0;

extern "C" cudaError_t cudaGetDevice(int* d) {
  *d = device;
  return cudaSuccess;
}
extern "C" cudaError_t cudaFuncSetAttribute(const void*, cudaFuncAttribute, int) {
  ++raised;
  return fail ? cudaErrorInvalidValue : cudaSuccess;
}

static char kernels[400 * 16];

static void expect(int got, int want, const char* what) {
  if (got != want) {
    std::printf("%s: %d, not %d\n", what, got, want);
    std::exit(1);
  }
}

static void every(int count) {
  for (int i = 0; i < count; ++i)
    if (mo::allow_smem(kernels + 16 * i, 1024) != cudaSuccess) std::exit(2);
}

static void run() {
  raised = 0;
  every(200);
  expect(raised, 200, "first calls");
  every(200);
  every(200);
  expect(raised, 200, "calls again");
}

int main() {
  run();
  std::thread(run).join();   // (a thread asks for itself)
  device = 1;
  raised = 0;
  every(200);
  every(200);
  expect(raised, 200, "another device");
  device = 0;
  every(200);
  expect(raised, 200, "the first device again");
  fail = 1;
  for (int i = 0; i < 2; ++i)
    if (mo::allow_smem(kernels + 16 * 399, 1024) == cudaSuccess) return 3;
  expect(raised, 202, "failures are not remembered");
  fail = 0;
  device = 2;                // more than there is room for: slower, and right
  raised = 0;
  for (; device < 8; ++device) every(400);
  if (raised < 6 * 400) return 4;
  std::puts("ok");
  return 0;
}
