// Host program of test_launch.py: the choice of a cluster size with the runtime's answers made up here.
// It makes no call that needs a GPU.
#include <cuda_runtime.h>

#include <cstdio>

static int g_answer[17], g_calls;  // clusters at once by blocks a cluster; below 0: the query fails
template <class K>
static cudaError_t fake_query(int* n, K, const cudaLaunchConfig_t* cfg) {
  ++g_calls;
  const int x = g_answer[cfg->gridDim.x];
  if (x < 0) return cudaErrorUnknown;
  *n = x;
  return cudaSuccess;
}
#define cudaOccupancyMaxActiveClusters fake_query
#define cudaGetLastError() cudaSuccess
#include "launch.cuh"

template <int I>
__global__ void kernel() {}

static int failed = 0;
static void expect(const char* what, long got, long want) {
  if (got != want) {
    printf("%s: %ld, not %ld\n", what, got, want);
    failed = 1;
  }
}
static void answers(int portable, int larger) {
  for (int i = 1; i <= 16; ++i) g_answer[i] = i <= 8 ? portable : larger;
}

template <int I>
static int choose(long units, long n, int narrowest = 1) {
  return tfd_host::cheapest_cluster(
      units, [](int i) { return tfd_host::clusters_at_once<kernel<I>>(0, i, 256, 0); },
      [&](int i) { return i >= narrowest; },
      [&](int i, int64_t rounds) { return rounds * (4096 + 64 * i + n / i); });
}

int main() {
  // one long row: the widest cluster is the cheapest, as far as the device can place it
  answers(20, 10);
  expect("all sizes", choose<0>(1, 1 << 20), 16);
  answers(20, 0);
  expect("none above 8", choose<1>(1, 1 << 20), 8);
  expect("a size that cannot be placed", tfd_host::clusters_at_once<kernel<1>>(0, 16, 256, 0), 0);
  answers(20, -1);
  expect("queries above 8 fail", choose<2>(1, 1 << 20), 8);
  answers(-1, -1);
  expect("all queries fail", choose<3>(1, 1 << 20), 8);
  expect("and only 16 would hold it", choose<3>(1, 1 << 20, 16), 16);
  answers(20, 0);
  expect("only 16 would hold it, which does not exist", choose<4>(1, 1 << 20, 16), 0);

  // an answer is asked for once, also that there is none; a failure is not kept
  g_calls = 0;
  expect("kept 0", tfd_host::clusters_at_once<kernel<1>>(0, 16, 256, 0), 0);
  expect("calls for it", g_calls, 0);
  answers(-1, -1);
  expect("failure", tfd_host::clusters_at_once<kernel<5>>(0, 4, 256, 0), -1);
  answers(20, 10);
  expect("the next time", tfd_host::clusters_at_once<kernel<5>>(0, 4, 256, 0), 20);
  answers(7, 7);
  expect("kept", tfd_host::clusters_at_once<kernel<5>>(0, 4, 256, 0), 20);
  expect("another device's", tfd_host::clusters_at_once<kernel<5>>(1, 4, 256, 0), 7);
  expect("no such device", tfd_host::clusters_at_once<kernel<5>>(-1, 4, 256, 0), -1);
  return failed;
}
