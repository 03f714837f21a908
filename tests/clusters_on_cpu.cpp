// The tables of clusters that a kernel has at work at a time (mx_plan.h): failures are not kept.
#include <cassert>
#include <cstdio>

#include "mx_plan.h"

int main() {
  static qgemv::MxClusterTable a, b;
  int asked = 0;
  auto answer = [&](int n) { return [&asked, n](int* to) { ++asked, *to = n; return true; }; };
  auto fail = [&](int* to) { ++asked, *to = 7; return false; };
  assert(a.get(3, 0, fail) == 0 && a.get(3, 0, fail) == 0 && asked == 2);  // asked again
  assert(a.get(3, 0, answer(15)) == 15 && asked == 3);
  assert(a.get(3, 0, fail) == 15 && a.get(3, 0, answer(9)) == 15 && asked == 3);  // and kept
  assert(a.get(2, 0, answer(36)) == 36 && a.get(3, 1, answer(14)) == 14 && a.get(3, 63, answer(13)) == 13);
  assert(a.get(1, 0, answer(0)) == 0 && a.get(1, 0, answer(5)) == 0 && asked == 7);  // none is an answer too
  assert(b.get(3, 0, answer(11)) == 11 && a.get(3, 0, fail) == 15 && asked == 8);  // another kernel's
  std::puts("done");
}
