// Host check of allow_smem with stand-ins for the three HIP calls: leave is
// asked for once per kernel and device, again after a failure, and never for
// 64 KiB or less.
#include <cstdio>

#include "wq_smem.hpp"

static int device = 0, asked = 0;
static hipError_t answer = hipSuccess;

extern "C" hipError_t hipGetDevice(int* d) {
  *d = device;
  return hipSuccess;
}
extern "C" hipError_t hipFuncSetAttribute(const void*, hipFuncAttribute, int) {
  ++asked;
  return answer;
}

static void kernel() {}

static int line(int n, bool ok) {
  if (!ok) std::printf("check %d failed: asked %d times\n", n, asked);
  return !ok;
}

int main() {
  int bad = 0;
  wq::SmemAllowed done{0}, other{0};
  auto call = [&](int dev, int bytes, wq::SmemAllowed& d) {
    device = dev;
    return wq::allow_smem(kernel, bytes, d);
  };
  bad += line(1, call(0, 65536, done) == hipSuccess && asked == 0);
  answer = hipErrorInvalidValue;
  bad += line(2, call(0, 90000, done) == hipErrorInvalidValue && asked == 1);
  answer = hipSuccess;
  bad += line(3, call(0, 90000, done) == hipSuccess && asked == 2);
  bad += line(4, call(0, 90000, done) == hipSuccess && asked == 2);
  bad += line(5, call(1, 90000, done) == hipSuccess && asked == 3);  // another GPU of the process
  bad += line(6, call(1, 90000, done) == hipSuccess && call(0, 90000, done) == hipSuccess && asked == 3);
  bad += line(7, call(0, 90000, other) == hipSuccess && asked == 4);
  bad += line(8, call(64, 90000, done) == hipSuccess && call(64, 90000, done) == hipSuccess && asked == 6);
  return bad;
}
