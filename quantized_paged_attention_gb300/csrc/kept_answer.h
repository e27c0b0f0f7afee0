// A number that has to be asked for, and asking may fail (host code).
#pragma once
#include <atomic>

namespace qpa {

// The number that ask(int*) gives, in `value`: asked until it answers once, then kept in `kept` (0: no answer yet, and never
// one). A failure is returned and nothing kept of it: it may have been the moment's, and the next call asks again.
template <class Ask>
auto kept_answer(std::atomic<int>& kept, Ask ask, int& value) -> decltype(ask(&value)) {
  decltype(ask(&value)) status{};           // (0: success)
  value = kept.load(std::memory_order_relaxed);
  if (value != 0) return status;
  status = ask(&value);
  if (status == decltype(status){}) kept.store(value, std::memory_order_relaxed);
  return status;
}

}  // namespace qpa
