// Loads and stores of row pieces (csrc/pieces.hpp) on the host, under
// AddressSanitizer: every piece of arrays of every length ending at any element, from
// buffers that hold the array and nothing more.  The device builtins and helpers that
// pieces.hpp takes from its neighbours are replaced by the host forms in device.hpp
// beside this file's copy.  Exits non-zero on the first mismatch.
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include "pieces.hpp"

using namespace qgemv;

static int g_fail = 0;

template <typename T, int N>
static void check(const char* what) {
  for (int64_t total = 1; total <= 41; ++total) {
    const size_t bytes = total * sizeof(T);
    unsigned char* const src = static_cast<unsigned char*>(malloc(bytes));  // (16-byte aligned)
    unsigned char* const dst = static_cast<unsigned char*>(malloc(bytes));  // (16-byte aligned)
    for (size_t i = 0; i < bytes; ++i) src[i] = (unsigned char)(37 * i + 11);
    for (int64_t e = 0; e < total; ++e)
      for (int count = 1; count <= N && e + count <= total; ++count) {
        const Bits<T, N> b = load_bits<T, true, N>(reinterpret_cast<const T*>(src), e, count, total);
        unsigned char want[sizeof(b.w)] = {};
        memcpy(want, src + e * sizeof(T), count * sizeof(T));
        memset(dst, 0xA5, bytes);
        store_bits<T, true, N>(reinterpret_cast<T*>(dst), e, count, b);
        bool ok = memcmp(want, b.w, sizeof(want)) == 0;
        for (size_t i = 0; i < bytes; ++i) {
          const bool in = i >= e * sizeof(T) && i < (e + count) * sizeof(T);
          ok = ok && dst[i] == (in ? src[i] : 0xA5);
        }
        if (!ok) {
          fprintf(stderr, "%s: %d elements at %d of %d\n", what, count, (int)e, (int)total);
          g_fail = 1;
        }
      }
    free(src);
    free(dst);
  }
}

int main() {
  check<_Float16, 8>("16-bit");
  check<float, 8>("fp32, 8");
  check<float, 4>("fp32, 4");
  if (!g_fail) printf("pieces: ok\n");
  return g_fail;
}
