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

// Where a token's rows lie; a wave finds it.
constexpr long long kNotHeld = -1, kNoSequence = -2;
struct Place {
  int row;               // in its sequence
  long long at;          // of head 0 in the layer's K or V, as (plane, head, column) counts; kNotHeld: not to
};                       // be touched (a status, a bad page); kNoSequence

// What finding it reads first, so that a kernel can ask for it ahead of its data
// (loads come back in order): the end column, and the first 64 sequences' state.  What
// is absent is read from where something is, since a branch would end in a wait.
struct Early {
  int E, lo, hi, n;
};
__device__ inline Early early_of(const TokenRows &P, int t) {
  const int32_t *any = P.c.kv_len;
  const int i = min(static_cast<int>(threadIdx.x & (kWave - 1)), P.B - 1);
  Early e;
  e.E = *(P.c.table ? any : P.c.end_col);
  e.lo = *(P.cu ? P.cu + i : any);
  e.hi = *(P.cu ? P.cu + i + 1 : any);
  e.n = P.c.kv_len[P.cu ? i : t / max(P.N, 1)];
  return e;
}

__device__ inline Place place_of(const TokenRows &P, int t, const Early &early) {
  const int lane = threadIdx.x & (kWave - 1), E = P.c.table ? 0 : early.E;
  int b = -1, t0 = 0, t1 = 0, n = early.n;
  if (P.cu) {
    // the first sequence that holds token t, with no fall before it
    for (int b0 = 0; b0 < P.B; b0 += kWave) {
      const bool is = b0 + lane < P.B;
      const int i = min(b0 + lane, P.B - 1), lo = b0 ? P.cu[i] : early.lo, hi = b0 ? P.cu[i + 1] : early.hi;
      const uint64_t who = __ballot(is && lo <= t && t < hi), falls = __ballot(is && lo > hi);
      if (who | falls) {
        const int l = __ffsll(static_cast<unsigned long long>(who | falls)) - 1;
        if (who >> l & 1) {
          b = b0 + l;
          t0 = read_lane(lo, l);
          t1 = read_lane(hi, l);
          n = b0 ? P.c.kv_len[b] : read_lane(early.n, l);
        }
        break;
      }
    }
    if (b < 0) return Place{0, kNoSequence};
  } else {
    b = t / P.N;
  }
  const Span s = span_of(P, b, t0, t1, n, E);
  const int row = s.row0 + (t - s.t0);
  if (s.st) return Place{row, kNotHeld};
  int plane = b, col = E - n + row;
  if (P.c.table) {
    const int i = cache_page(P.c, row);
    plane = P.c.table[static_cast<long long>(b) * P.c.max_pages + i];
    col = row - i * P.c.cols;
    if (plane < 0 || plane >= P.c.planes) return Place{row, kNotHeld};
  }
  return Place{row, static_cast<long long>(plane) * P.c.H * P.c.cols + col};
}

}  // namespace
}  // namespace specv
