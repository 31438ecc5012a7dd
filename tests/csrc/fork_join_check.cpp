// Test helper: runs librpa's order of two parts on two streams (fork_join.h)
// with steps that only note their letter and fail where asked.  Built by the
// test suite only; not part of the library.
#include "fork_join.h"

// `fails`: bit i makes step i (fork, there, mark, here, join) return 10 + i.
// `order`: receives the letters of the steps that ran, and a zero.
extern "C" int fork_join_check(unsigned fails, char* order) {
  auto step = [&](int i, char letter) {
    return [=, &order] {
      *order++ = letter;
      return fails >> i & 1u ? 10 + i : 0;
    };
  };
  const int err = rpa::fork_join(step(0, 'f'), step(1, 't'), step(2, 'm'), step(3, 'h'), step(4, 'j'));
  *order = 0;
  return err;
}
