"""CPU checks of csrc/form_buffers.h, the growth of an engine's attention-form buffers, with memory that
the test hands out (and refuses)."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
#include "form_buffers.h"
#include <cstdio>
#include <cstdlib>
#include <map>
#include <vector>

#define CHECK(c) do { if (!(c)) { std::printf("line %d: %s\n", __LINE__, #c); std::exit(1); } } while (0)

struct Memory {
  std::map<void*, size_t> held;
  int allocs = 0, refuse = -1;  // refuse: the allocation of that number fails
  int settled = 0;
  bool busy = true;             // queued work uses what was there before
  void* alloc(size_t n) {
    if (allocs++ == refuse) return nullptr;
    void* p = std::malloc(1);
    held[p] = n;
    return p;
  }
  void settle() { ++settled; busy = false; }
  void release(void* p) {
    CHECK(held.count(p));
    CHECK(!busy || fresh.count(p));
    held.erase(p);
    std::free(p);
  }
  std::map<void*, int> fresh;
  size_t bytes() const { size_t n = 0; for (auto& h : held) n += h.second; return n; }
};

int main() {
  for (size_t n = 1; n < 100000; ++n) {
    const size_t q = quarter_octave(n);
    CHECK(q >= n && q <= n + n / 4 + 1 && quarter_octave(q) == q);
  }
  auto sums = [](int max_kv) { return (size_t)max_kv * 100; };
  const long long most = 50000;
  {  // grows with the longest row, within the arena's positions; counts what it holds
    Memory m;
    FormBuffers b;
    int grown = 0;
    for (int n = 1; n <= 50000; n += 7) {
      m.busy = true;
      const int before = m.settled;
      CHECK(grow_form(&b, n, most, 128, 8, sums, m));
      grown += m.settled - before;
      CHECK(b.max_kv >= n && b.max_kv <= most && b.max_pages * 128 >= b.max_kv);
      CHECK(n < 1024 || b.max_kv <= n + n / 4 + 1);
      CHECK(b.table_bytes >= (size_t)8 * b.max_pages * 4 && b.ws_bytes >= sums(b.max_kv));
      CHECK(m.held.size() == 2 && m.bytes() == b.table_bytes + b.ws_bytes);
    }
    CHECK(grown > 10 && grown < 50);
    // a call of more rows wants more sums alone; a smaller one nothing
    void* table = b.table;
    const int kv = b.max_kv;
    CHECK(grow_form(&b, 10, most, 128, 8, [](int n) { return (size_t)n * 1000; }, m));
    CHECK(b.table == table && b.max_kv == kv && b.ws_bytes >= (size_t)kv * 1000);
    const int before = m.settled;
    CHECK(grow_form(&b, kv, most, 128, 8, sums, m) && m.settled == before);
  }
  {  // no sums at all
    Memory m;
    FormBuffers b;
    CHECK(grow_form(&b, 5, most, 128, 8, [](int) { return (size_t)0; }, m));
    CHECK(!b.ws && b.ws_bytes == 0 && b.table && m.held.size() == 1);
  }
  for (int which = 0; which < 2; ++which) {  // the table's, or the sums', memory is refused
    Memory m;
    FormBuffers b;
    CHECK(grow_form(&b, 1500, most, 128, 8, sums, m));
    const FormBuffers was = b;
    m.busy = true;
    m.allocs = 0;
    m.refuse = which;
    // (what grow_form itself has just got it may give back while work is queued)
    struct Fresh : Memory {
      Memory* m;
      void* alloc(size_t n) { void* p = m->alloc(n); if (p) m->fresh[p] = 1; return p; }
      void settle() { m->settle(); }
      void release(void* p) { m->release(p); }
    } f;
    f.m = &m;
    const int before = m.settled;
    CHECK(!grow_form(&b, 20000, most, 128, 8, sums, f));
    CHECK(m.settled == before);  // nothing was waited for, no step dropped
    CHECK(b.max_kv == was.max_kv && b.max_pages == was.max_pages && b.table == was.table && b.ws == was.ws);
    CHECK(b.table_bytes == was.table_bytes && b.ws_bytes == was.ws_bytes);
    CHECK(m.held.size() == 2 && m.bytes() == b.table_bytes + b.ws_bytes);
    // shorter rows go on, and longer ones once there is memory
    CHECK(grow_form(&b, 1500, most, 128, 8, sums, m) && m.settled == before);
    m.refuse = -1;
    CHECK(grow_form(&b, 20000, most, 128, 8, sums, m) && b.max_kv >= 20000);
    CHECK(m.held.size() == 2);
  }
  {  // the first call of all is refused
    Memory m;
    FormBuffers b;
    m.refuse = 1;
    m.busy = false;
    CHECK(!grow_form(&b, 10, most, 128, 8, sums, m));
    CHECK(m.held.empty());
    FormBuffers none;
    CHECK(b.max_kv == none.max_kv && !b.table && !b.ws);
  }
  std::puts("ok");
}
"""


def test_growth(tmp_path):
    src, exe = tmp_path / "grow.cc", tmp_path / "grow"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-I",
                    os.path.join(ROOT, "continuous_batching_transformer_gb300", "csrc"), str(src), "-o", str(exe)],
                   check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert (r.returncode, r.stdout) == (0, "ok\n"), r.stdout + r.stderr
