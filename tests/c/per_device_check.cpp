// csrc/per_device.h: answers are kept per device and index, failures are not kept.
#include <cstdio>

#include "per_device.h"

static int failures = 0;
static void expect(int got, int want, const char* what) {
  if (got != want) {
    ++failures;
    std::printf("%s: got %d, want %d\n", what, got, want);
  }
}

int main() {
  static moe_host::PerDevice<3> t;
  int asked = 0;
  auto says = [&](int v) { return [&asked, v] { ++asked; return v; }; };
  expect(t.get(0, 1, 9, says(152)), 152, "first answer");
  expect(t.get(0, 1, 9, says(1)), 152, "kept");
  expect(t.get(1, 1, 9, says(132)), 132, "another device");
  expect(t.get(0, 2, 9, says(120)), 120, "another index");
  expect(asked, 3, "queries");
  expect(t.get(2, 0, 9, says(0)), 9, "a failure's fallback");
  expect(t.get(2, 0, 9, says(148)), 148, "asked again after a failure");
  expect(t.get(-1, 0, 9, says(7)), 7, "unknown device");
  expect(t.get(-1, 0, 9, says(8)), 8, "unknown device is not kept");
  expect(t.get(64, 2, 9, says(-1)), 9, "device past the table");
  std::printf("ok: %d failure(s)\n", failures);
  return failures != 0;
}
