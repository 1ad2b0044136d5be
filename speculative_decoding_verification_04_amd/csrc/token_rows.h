// Tokens of a call and their rows in the cache (gfx950): shared by the calls that
// write and read rows token by token.
//
// Either B sequences of N tokens each, which become (or are) rows n_b .. n_b + N - 1,
// or packed ranges [cu[b], cu[b + 1]), which are sequence b's last rows.
#pragma once

#include "cache_view.h"

namespace specv {
namespace {

struct TokenRows {
  CacheView c;
  int T, B, N;               // N 0: packed
  const int32_t *cu;
  int32_t *status;
};

// A sequence's new tokens and where their rows start.
struct Span {
  int t0, len, row0;   // first token, tokens, first row
  int st;              // status bits; nonzero: nothing is written to the cache
};

// t0, t1: the sequence's token range (packed calls); n: its length; E: the
// rectangle's end (pages: 0).
__device__ inline Span span_of(const TokenRows &P, int b, int t0, int t1, int n, int E) {
  Span s;
  s.st = 0;
  if (P.cu) {
    // no difference is taken before its operands are known to be in range
    const bool in = t0 >= 0 && t0 <= t1 && t1 <= P.T;
    s.t0 = in ? t0 : 0;
    s.len = in ? t1 - t0 : 0;
    if (!in || n < s.len) s.st = SPEC_ST_BAD_STATE;
    s.row0 = s.st ? 0 : n - s.len;
  } else {
    s.t0 = b * P.N;
    s.len = P.N;
    s.row0 = n;
    if (n < 0) s.st = SPEC_ST_BAD_STATE;
  }
  const long long cap = cache_capacity(P.c), end = static_cast<long long>(n) + (P.cu ? 0 : P.N);
  if (P.c.table) {
    if (end > cap) s.st |= SPEC_ST_CAPACITY;
  } else {
    if (E < 0 || static_cast<long long>(E) + (P.cu ? 0 : P.N) > cap) s.st |= SPEC_ST_CAPACITY;
    if (n > E) s.st |= SPEC_ST_BAD_STATE;
  }
  return s;
}

// The status of one sequence per wave: its span and the pages of its new rows.
__device__ inline void write_status(const TokenRows &P, int b) {
  const int lane = threadIdx.x & (kWave - 1);
  if (b >= P.B) return;
  const Span s = span_of(P, b, P.cu ? P.cu[b] : 0, P.cu ? P.cu[b + 1] : 0, P.c.kv_len[b], P.c.table ? 0 : *P.c.end_col);
  int st = s.st;
  if (P.cu) {
    bool falls = false;                                   // before the sequence
    for (int i = lane; i < b; i += kWave) falls |= P.cu[i] > P.cu[i + 1];
    if (__any(falls)) st |= SPEC_ST_BAD_STATE;
  }
  if (!st && P.c.table && s.len > 0) {
    bool bad = false;
    const int last = cache_page(P.c, s.row0 + s.len - 1);
    for (int i = cache_page(P.c, s.row0) + lane; i <= last; i += kWave) {
      const int page = P.c.table[static_cast<long long>(b) * P.c.max_pages + i];
      bad |= page < 0 || page >= P.c.planes;
    }
    if (__any(bad)) st = SPEC_ST_BAD_STATE;
  }
  if (lane == 0) P.status[b] = st;
}

}  // namespace
}  // namespace specv
