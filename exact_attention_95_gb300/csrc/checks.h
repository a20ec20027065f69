// checks.h -- argument checks that several files of entry points share.
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace attn {

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Whether one of the first `written` of `count` arrays shares a byte with another.
struct Span {
  const void* p;
  size_t n;  // bytes
};
inline bool overlap(const Span& a, const Span& b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return a.n > 0 && b.n > 0 && x < y + b.n && y < x + a.n;
}
inline bool any_overlap(const Span* a, int written, int count) {
  for (int i = 0; i < written; ++i)
    for (int j = i + 1; j < count; ++j)
      if (overlap(a[i], a[j])) return true;
  return false;
}

// Rows of d contiguous elements of `size` bytes, one for each of B x H x N;
// strides in elements (those of dimensions of one are not looked at).
struct Rows {
  const void* p;
  int64_t n[3], stride[3];  // batch, head, token
  int64_t d, size;

  Rows(const void* p_, int64_t B, int64_t H, int64_t N, int64_t batch, int64_t head, int64_t token, int64_t d_, int size_)
      : p(p_), n{B, H, N}, stride{B > 1 ? batch : 0, H > 1 ? head : 0, N > 1 ? token : 0}, d(d_), size(size_) {}
  // Elements from the first to behind the last.
  int64_t extent() const { return (n[0] - 1) * stride[0] + (n[1] - 1) * stride[1] + (n[2] - 1) * stride[2] + d; }
  Span span() const { return {p, (size_t)(extent() * size)}; }
  // Strides of whole 16 bytes, none negative or past what a 64-bit offset holds.
  bool strides_ok() const {
    for (int i = 0; i < 3; ++i)
      if (stride[i] < 0 || stride[i] * size % 16 != 0 || stride[i] > (int64_t(1) << 40) || n[i] > (int64_t(1) << 31)) return false;
    const double top = (double)(n[0] - 1) * stride[0] + (double)(n[1] - 1) * stride[1] + (double)(n[2] - 1) * stride[2];
    return top < 1e18;
  }
  // Whether no two of the rows share an element: by increasing stride, each
  // dimension steps over all that lies below it.
  bool distinct() const {
    int at[3] = {0, 1, 2};
    for (int i = 0; i < 2; ++i)
      for (int j = 0; j < 2 - i; ++j)
        if (stride[at[j]] > stride[at[j + 1]]) {
          const int t = at[j];
          at[j] = at[j + 1];
          at[j + 1] = t;
        }
    int64_t below = d;
    for (int i : at) {
      if (n[i] == 1) continue;
      if (stride[i] < below) return false;
      below += (n[i] - 1) * stride[i];
    }
    return true;
  }
  bool same(const Rows& o) const {
    for (int i = 0; i < 3; ++i)
      if (n[i] != o.n[i] || stride[i] != o.stride[i]) return false;
    return p == o.p && d == o.d && size == o.size;
  }
  // Elements from a token's first to behind its last, where its heads lie
  // between one token and the next and batches whole tokens apart; else 0.
  int64_t token_width(int64_t token) const {
    const int64_t w = (n[1] - 1) * stride[1] + d;
    return w <= token && (n[2] == 1 || stride[2] == token) && stride[0] % token == 0 ? w : 0;
  }
};
// Distances that rows of two sets have in common: `stride` times a number from lo to hi.
struct Steps {
  int64_t stride, lo, hi;
};
// Whether off plus one of each of the steps' distances is less than d away from 0; true also where that
// takes more than `tries` tries to tell.  With strides that step over what lies below them, as those of a
// packed array do, each step has two or three candidates.
inline bool may_meet(int64_t off, const Steps* s, int count, int64_t d, int& tries) {
  if (--tries < 0) return true;
  if (count == 0) return off > -d && off < d;
  int64_t low = 0, high = 0;  // of the steps behind this one
  for (int i = 1; i < count; ++i) {
    low += s[i].stride * s[i].lo;
    high += s[i].stride * s[i].hi;
  }
  // off + stride * n + (low .. high) has to reach into (-d, d).
  const int64_t from = -d + 1 - off - high, to = d - 1 - off - low, a = s[0].stride;
  const int64_t first = from / a + (from % a > 0), last = to / a - (to % a < 0);
  for (int64_t n = first > s[0].lo ? first : s[0].lo; n <= (last < s[0].hi ? last : s[0].hi); ++n)
    if (may_meet(off + a * n, s + 1, count - 1, d, tries)) return true;
  return false;
}
// Whether two sets of rows certainly share no element: their spans do not meet, or
// both have their tokens' heads side by side in the same packed array (slices of
// a projection), in parts of a token that do not meet, or no distance between their rows is
// less than a row.
inline bool apart(const Rows& a, const Rows& b) {
  if (!overlap(a.span(), b.span())) return true;
  if (a.size != b.size || a.d != b.d) return false;
  const int64_t bytes = (int64_t)(reinterpret_cast<intptr_t>(b.p) - reinterpret_cast<intptr_t>(a.p));
  if (bytes % a.size) return false;
  const int64_t token = a.n[2] > 1 ? a.stride[2] : b.n[2] > 1 ? b.stride[2] : a.n[0] > 1 ? a.stride[0] : b.stride[0];
  if (token > 0) {
    const int64_t wa = a.token_width(token), wb = b.token_width(token);
    const int64_t off = ((bytes / a.size) % token + token) % token;  // of b's part behind a's, within a token
    if (wa && wb && off >= wa && off + wb <= token) return true;
  }
  Steps s[6];
  int count = 0;
  for (int k = 0; k < 6; ++k) {
    const Rows& r = k < 3 ? a : b;
    const int64_t stride = r.stride[k % 3], most = r.n[k % 3] - 1;
    if (most == 0 || stride == 0) continue;
    int at = 0;
    while (at < count && s[at].stride > stride) ++at;
    if (at == count || s[at].stride != stride) {
      for (int i = count++; i > at; --i) s[i] = s[i - 1];
      s[at] = {stride, 0, 0};
    }
    (k < 3 ? s[at].lo : s[at].hi) += k < 3 ? -most : most;
  }
  int tries = 4096;
  return !may_meet(bytes / a.size, s, count, a.d, tries);
}

}  // namespace attn
