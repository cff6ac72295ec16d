// Host-side check of allow_smem (compiled and run by tests/test_smem_limit.py;
// no GPU needed): two threads ask for different sizes of one kernel, and the
// call that sets the limit is a fake that holds the larger request back until
// the smaller one has been made, or 300 ms have passed.  Whatever the order, the
// kernel's limit must not be below what a later launch is let through with.
#include <chrono>
#include <condition_variable>
#include <cstdio>
#include <mutex>
#include <thread>

#include "w4a_internal.h"

static std::mutex mu;
static std::condition_variable cv;
static int limit = 48 * 1024, small_done = 0, big_inside = 0, calls = 0;
static cudaError_t answer = cudaSuccess;
constexpr int BIG = 164 * 1024, SMALL = 57 * 1024;

extern "C" cudaError_t cudaGetDevice(int* d) {
  *d = 0;
  return cudaSuccess;
}
extern "C" cudaError_t cudaFuncSetAttribute(const void*, cudaFuncAttribute, int bytes) {
  std::unique_lock<std::mutex> lk(mu);
  ++calls;
  if (answer != cudaSuccess) return answer;
  limit = bytes;
  if (bytes == BIG) {
    big_inside = 1;
    cv.notify_all();
    cv.wait_for(lk, std::chrono::milliseconds(300), [] { return small_done != 0; });
  }
  return cudaSuccess;
}

static int fails = 0;
#define CHECK(c)                                      \
  do {                                                \
    if (!(c)) {                                       \
      ++fails;                                        \
      printf("FAIL line %d: %s\n", __LINE__, #c);     \
    }                                                 \
  } while (0)

int main() {
  using namespace w4a;
  static SmemMark mark;
  const void* fn = &mark;
  std::thread a([&] { CHECK(allow_smem(fn, BIG, mark) == cudaSuccess); });
  std::thread b([&] {
    {
      std::unique_lock<std::mutex> lk(mu);
      cv.wait_for(lk, std::chrono::seconds(5), [] { return big_inside != 0; });
    }
    CHECK(allow_smem(fn, SMALL, mark) == cudaSuccess);
    std::lock_guard<std::mutex> lk(mu);
    small_done = 1;
    cv.notify_all();
  });
  a.join();
  b.join();
  // a launch of a size between the two, by either thread's leave
  CHECK(allow_smem(fn, 100 * 1024, mark) == cudaSuccess);
  CHECK(limit >= BIG);

  // a size that the kernel has is not asked for again; one that was refused is
  const int before = calls;
  CHECK(allow_smem(fn, 90 * 1024, mark) == cudaSuccess && calls == before);
  answer = cudaErrorInvalidValue;
  CHECK(allow_smem(fn, 200 * 1024, mark) == cudaErrorInvalidValue);
  CHECK(allow_smem(fn, 200 * 1024, mark) == cudaErrorInvalidValue && calls == before + 2);
  answer = cudaSuccess;
  CHECK(allow_smem(fn, 200 * 1024, mark) == cudaSuccess && limit == 200 * 1024);
  CHECK(allow_smem(fn, 16 * 1024, mark) == cudaSuccess && limit == 200 * 1024);  // fits the default
  if (!fails) printf("smem ok\n");
  return fails != 0;
}
