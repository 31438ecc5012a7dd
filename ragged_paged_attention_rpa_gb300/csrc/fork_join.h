// Two parts of a call on two streams: the order of the steps and what an error
// in one of them leaves out.
#pragma once

namespace rpa {

// fork: the side stream waits for everything enqueued on the caller's so far;
// there: a part on the side stream; mark: the join event behind it; here: the
// other part on the caller's stream; join: the caller's stream waits for the
// event.  Each returns 0 or an error; the first one is returned.  From the fork
// on the side stream is joined whatever failed: a part that ended in an error
// may have enqueued some of its kernels, which still write the caller's buffers,
// and a capture must not be left with a stream that is not joined.
template <typename Fork, typename There, typename Mark, typename Here, typename Join>
int fork_join(Fork&& fork, There&& there, Mark&& mark, Here&& here, Join&& join) {
  if (const int err = fork()) return err;
  int err = there();
  const int unmarked = mark();
  if (err == 0) err = unmarked;
  if (err == 0) err = here();
  if (unmarked == 0) {
    const int unjoined = join();
    if (err == 0) err = unjoined;
  }
  return err;
}

}  // namespace rpa
