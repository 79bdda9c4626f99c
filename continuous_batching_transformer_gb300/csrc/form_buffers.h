// form_buffers.h -- the two device buffers that an engine's attention form grows with its rows: the
// calls' page table and the attention's workspace.  Plain host code; the memory is the caller's to get.
#pragma once
#include <algorithm>
#include <cstddef>
#include <cstdint>

struct FormBuffers {
  int max_kv = 0;     // the longest row that the calls' bounds allow
  int max_pages = 0;  // and its pages: the table's row
  void* table = nullptr;
  size_t table_bytes = 0;
  void* ws = nullptr;
  size_t ws_bytes = 0;
};

// n rounded up to four steps an octave: a growing size passes few of them, and none holds more than a
// quarter too much
inline size_t quarter_octave(size_t n) {
  size_t step = 1;
  while (n > 8 * step) step *= 2;
  return (n + step - 1) / step * step;
}

// Makes b fit rows of up to `longest` positions, of at most `most`, in a table of `rows` rows, and a
// workspace of ws_bytes(max_kv) bytes.  mem.alloc(bytes) gives memory or NULL; mem.settle() makes sure
// that nothing uses the buffers or bounds of before any more, mem.release(p) gives memory back.
// Where memory is lacking, b is left as it was, so that shorter rows can go on, and false returned.
template <class Mem, class WsBytes>
bool grow_form(FormBuffers* b, long long longest, long long most, int page, int rows, const WsBytes& ws_bytes,
               Mem& mem) {
  FormBuffers n = *b;
  if (longest > n.max_kv) {
    const long long want = (long long)quarter_octave((size_t)std::max<long long>(longest, 1024));
    n.max_kv = (int)std::min(want, std::max(longest, most));
    n.max_pages = (int)(((long long)n.max_kv + page - 1) / page);
    n.table_bytes = std::max(n.table_bytes, (size_t)rows * n.max_pages * sizeof(int32_t));
  }
  const size_t need = ws_bytes(n.max_kv);
  if (need > n.ws_bytes) n.ws_bytes = quarter_octave(need);
  if (n.max_kv == b->max_kv && n.ws_bytes == b->ws_bytes) return true;
  const bool table = n.table_bytes > b->table_bytes, ws = n.ws_bytes > b->ws_bytes;
  if (table && !(n.table = mem.alloc(n.table_bytes))) return false;
  if (ws && !(n.ws = mem.alloc(n.ws_bytes))) {
    if (table) mem.release(n.table);
    return false;
  }
  mem.settle();
  if (table && b->table) mem.release(b->table);
  if (ws && b->ws) mem.release(b->ws);
  *b = n;
  return true;
}
