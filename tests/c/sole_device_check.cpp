// Whether the process sees one GPU alone, by fake answers of the device query.
#include <cstdio>

#include "per_device.h"

static int failures = 0;
#define CHECK(cond)                                       \
  do {                                                    \
    if (!(cond)) {                                        \
      std::printf("line %d: %s\n", __LINE__, #cond);      \
      ++failures;                                         \
    }                                                     \
  } while (0)

int main() {
  const auto answer = [](int devices, bool ok) {
    return [=](int* n) {
      *n = devices;
      return ok;
    };
  };
  CHECK(moe_host::sole_device(answer(1, true)));
  CHECK(!moe_host::sole_device(answer(2, true)));
  CHECK(!moe_host::sole_device(answer(8, true)));
  CHECK(!moe_host::sole_device(answer(0, true)));
  CHECK(!moe_host::sole_device(answer(1, false)));  // a query that failed says nothing
  return failures;
}
