// Causal attention of packed prompts over the cache (gfx950).
//
// The tokens of B sequences lie packed; sequence b's are tokens
// [cu[b], cu[b + 1]) and the last cu[b + 1] - cu[b] of its n_b cached rows are
// theirs (so a prompt may follow rows that are cached already).  Token i of
// len sees rows [0, n_b - len + i].
//
// Design.  Bound by the matrix cores: 4 D flops a visible pair against the
// 2 D bytes of a row, which a tile of 128 (or 64) query rows uses that often.  The
// lengths are on the device, so the grid is the largest that T tokens in B
// sequences can need, and a workgroup finds its (sequence, tile) from the
// sequences' tile counts.
// Measured: prompts of 12001 and 10147 tokens, 32 heads of 128 over 8 KV heads in
// bf16: 1.92 ms = 1050 TFLOP/s, where an 8192^3 product reaches 1172 (the matrix
// units are busy 56% of the cycles and the vector units, with the softmax, most
// of the others); 8 prompts of 256 .. 2048 tokens, 14 heads of 64 over pages: 50 us
// = 560 TFLOP/s, since heads of 64 halve the products but not the softmax; 4
// prompts of 23 .. 64 tokens in float32: 8 us, latency.
#include "attention.h"

namespace specv {
namespace {
using namespace attn;

struct Where {
  int b, tile, tiles;
};

// Tokens of the lane's sequence b (b past the last: 0); -1 where its range is not
// inside [0, T], or where cu falls there or before: it could hold other sequences'
// tokens.  Whole waves call it, for 64 sequences after the other.
__device__ inline int prompt_len(const Params &P, int b, bool &fallen) {
  const int i = min(b, P.B - 1), lo = P.cu[i], hi = P.cu[i + 1];
  const uint64_t falls = __ballot(b < P.B && lo > hi);
  const bool follows = !fallen && !(falls & (~0ull >> (kWave - 1 - (threadIdx.x & (kWave - 1)))));   // up to the own
  fallen |= falls != 0;
  return b >= P.B ? 0 : follows && lo >= 0 && hi <= P.T ? hi - lo : -1;
}
__device__ inline int prompt_status(const Params &P, int b, int len) {
  if (len < 0) return SPEC_ST_BAD_STATE;
  const int n = P.c.kv_len[b];
  int st = n < len ? SPEC_ST_BAD_STATE : 0;
  const long long cap = cache_capacity(P.c);
  if (P.c.table) {
    if (n > cap) st |= SPEC_ST_CAPACITY;
  } else {
    const int E = *P.c.end_col;
    if (E < 0 || E > cap) st |= SPEC_ST_CAPACITY;
    if (n > E) st |= SPEC_ST_BAD_STATE;
  }
  return st;
}

// The sequence and tile of flat tile number f.  Past the last: b = -1, the number
// among those that have no tile, and how many they are.
// Where the workgroups do not all fit the chip at once, up to 64 sequences' tiles
// are taken by their number, the highest (the longest walks) of all sequences
// first, so that no long walk starts late: 8 prompts of 256 .. 2048 tokens (14
// heads of 64) take 50 us and not 57.  Tiles numbered `level` and more are sum
// max(0, tiles_b - level), and the level of tile f is found by halving.  Else
// sequences follow each other, each from its last tile to its first.
template <int kTileRows>
__device__ inline Where find_tile(const Params &P, int f) {
  const int lane = threadIdx.x & (kWave - 1);
  bool fallen = false;
  auto tiles_of = [&](int b) {
    const int len = prompt_len(P, b, fallen);
    return len > 0 ? static_cast<int>((static_cast<long long>(len) * P.G + kTileRows - 1) / kTileRows) : 0;
  };
  if (P.B <= kWave && gridDim.x > 512) {
    const int tiles = tiles_of(lane);
    auto from = [&](int level) {
      return wave_reduce(max(0, tiles - level), [](int x, int y) { return x + y; });
    };
    if (from(0) <= f) return Where{-1, f - from(0), static_cast<int>(gridDim.x / P.c.H) - from(0)};
    int lo = 0, hi = wave_max_i(tiles);                   // from(lo) > f >= from(hi) = 0
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (from(mid) > f) lo = mid;
      else hi = mid;
    }
    uint64_t who = __ballot(tiles > lo);
    for (int skip = f - from(lo + 1); skip > 0; --skip) who &= who - 1;
    const int b = __ffsll(static_cast<unsigned long long>(who)) - 1;
    return Where{b, lo, read_lane(tiles, b)};
  }
  int base = 0;
  for (int b0 = 0; b0 < P.B; b0 += kWave) {
    const int tiles = tiles_of(b0 + lane);
    const int upto = wave_incl_scan(tiles);
    const uint64_t who = __ballot(base + upto > f);
    if (who) {
      const int l = __ffsll(static_cast<unsigned long long>(who)) - 1;
      const int n = read_lane(tiles, l);
      const int before = base + read_lane(upto, l) - n;
      return Where{b0 + l, n - 1 - (f - before), n};
    }
    base += read_lane(upto, kWave - 1);
  }
  return Where{-1, f - base, static_cast<int>(gridDim.x / P.c.H) - base};
}

// A range that reaches past the call's tokens has no tiles, and its sequence a
// status; the tokens that it does have get zeros, from the workgroups without a
// tile (the grid counts at least one for each such sequence): workgroup `which`
// of `of`.
template <typename T>
__device__ inline void zero_outside(const Params &P, long long which, long long of) {
  const int lane = threadIdx.x & (kWave - 1);
  const long long heads = static_cast<long long>(P.c.H) * P.G, row = heads * P.c.D * sizeof(T) / 16;
  for (int b0 = 0; b0 < P.B; b0 += kWave) {
    const int i = min(b0 + lane, P.B - 1), lo = P.cu[i], hi = P.cu[i + 1];
    const bool is = b0 + lane < P.B;
    const uint64_t falls = __ballot(is && lo > hi);       // no tokens from there on
    uint64_t outside = __ballot(is && (lo < 0 || hi > P.T));
    if (falls) outside &= (falls & -falls) - 1;
    for (; outside; outside &= outside - 1) {
      const int l = __ffsll(static_cast<unsigned long long>(outside)) - 1;
      const long long t0 = max(read_lane(lo, l), 0), t1 = min(read_lane(hi, l), P.T);
      u32x4 *out = reinterpret_cast<u32x4 *>(P.out);
      for (long long x = t0 * row + which * kThreads + threadIdx.x; x < t1 * row; x += of * kThreads) out[x] = u32x4{0, 0, 0, 0};
      if (P.lse)
        for (long long x = t0 * heads + which * kThreads + threadIdx.x; x < t1 * heads; x += of * kThreads) P.lse[x] = -INFINITY;
    }
    if (falls) return;
  }
}

template <typename T, int DP, int RW, bool PAGED>
__global__ __launch_bounds__(kThreads, DP <= 128 && sizeof(T) == 2 && RW > 1 ? 2 : 1) void prompt_kernel(Params P) {
  using S = Shape<T, DP, RW>;
  constexpr int kTileRows = 32 * RW;
  __shared__ __attribute__((aligned(16))) char buf0[S::kLds];
  __shared__ __attribute__((aligned(16))) char buf1[S::kLds];
  const int H = P.c.H;
  const int h = blockIdx.x % H, f = blockIdx.x / H;
  if (blockIdx.x == 0 && P.status && threadIdx.x < kWave) {
    // sequences without tokens have no tile that would report on them
    bool fallen = false;
    for (int b0 = 0; b0 < P.B; b0 += kWave) {
      const int b = b0 + threadIdx.x, len = prompt_len(P, b, fallen);
      if (b < P.B && len <= 0) P.status[b] = prompt_status(P, b, len);
    }
  }
  const Where w = find_tile<kTileRows>(P, f);
  if (w.b < 0) {
    zero_outside<T>(P, static_cast<long long>(w.tile) * H + h, static_cast<long long>(w.tiles) * H);
    return;
  }
  Job J;
  const int len = P.cu[w.b + 1] - P.cu[w.b], st = prompt_status(P, w.b, len), n = P.c.kv_len[w.b];
  J.b = w.b;
  J.h = h;
  J.row0 = w.tile * kTileRows;
  J.tokens = len;
  J.token0 = P.cu[w.b];
  J.limit0 = n - len + 1;
  J.total = n;
  const bool reports = P.status && h == 0 && w.tile == w.tiles - 1;   // the tile that walks every row
  if (st) {
    put_zeros<T>(P, J, kTileRows);
    if (reports && threadIdx.x == 0) P.status[w.b] = st;
    return;
  }
  J.start_col = PAGED ? 0 : *P.c.end_col - n;
  const int last = min((J.row0 + kTileRows - 1) / P.G, len - 1);      // the tile's last token
  J.t0 = 0;
  J.t1 = (J.limit0 + last + S::kKT - 1) / S::kKT;
  Done<DP, S::kKW> W;
  const bool bad = walk<T, DP, RW, PAGED, true, false>(P, J, W, buf0, buf1);
  put_rows<T>(P, J, W, true);
  if (reports && threadIdx.x == 0) P.status[w.b] = bad ? SPEC_ST_BAD_STATE : 0;
}

// Workgroups that T tokens in B sequences can need with rw waves side by side:
// each sequence rounds up once.
inline long long prompt_grid(int T, int B, int H, int G, int rw) {
  return (static_cast<long long>(T) * G / (32 * rw) + B) * H;
}

template <typename T, int DP, int RW>
int launch_rows(const Params &P, hipStream_t s) {
  const long long workgroups = prompt_grid(P.T, P.B, P.c.H, P.G, RW);
  if (!launchable(workgroups, kThreads)) return SPEC_EINVAL;
  const dim3 grid(static_cast<unsigned>(workgroups));
  (void)hipGetLastError();
  if (P.c.table)
    hipLaunchKernelGGL((prompt_kernel<T, DP, RW, true>), grid, dim3(kThreads), 0, s, P);
  else
    hipLaunchKernelGGL((prompt_kernel<T, DP, RW, false>), grid, dim3(kThreads), 0, s, P);
  return launch_status();
}

// Few rows take 64 to a workgroup, two waves behind each other: with fewer than
// 384 tiles of 128 the chip has workgroups to spare, and a tile's walk is
// shorter.  One prompt of 500 / 1000 / 2000 tokens (32 heads of 128, bf16): 14.2 /
// 25.3 / 62.3 us against 16.1 / 26.1 / 51.4 with 128 rows; 4 prompts of up to 400
// tokens (8 heads of 128, float32): 40 against 61.
template <typename T, int DP>
int launch_prompt(const Params &P, hipStream_t s) {
  if constexpr (sizeof(T) * DP <= 512) {
    if (static_cast<long long>(P.T) * P.G * P.c.H < 384 * 128) return launch_rows<T, DP, 2>(P, s);
  }
  return launch_rows<T, DP, 4>(P, s);
}

int prompt_call(const void *q, int64_t q_stride, const void *kv, spec_dtype dt, int L, int planes, int B, int H,
                int cols, int D, int layer, int T, int G, const int32_t *table, int max_pages, bool paged,
                const int32_t *end_col, const int32_t *kv_len, const int32_t *cu, float scale, void *out, float *lse,
                int32_t *status, spec_stream_t stream) {
  if (!cu) return SPEC_EINVAL;
  Params P;
  const int err = fill(P, q, q_stride, kv, dt, L, planes, B, H, cols, D, layer, G, table, max_pages, paged, end_col,
                       kv_len, scale, out, lse, status);
  if (err) return err;
  if (T < 1) return SPEC_EINVAL;
  if (static_cast<long long>(T) * G >= INT32_MAX) return SPEC_EINVAL;
  const size_t elt = dt == SPEC_BF16 ? 2 : 4, hd = static_cast<size_t>(H) * G * D, b4 = static_cast<size_t>(B) * 4;
  const void *ins[] = {q, kv, table, end_col, kv_len, cu};
  const size_t in_n[] = {((T - 1) * static_cast<size_t>(q_stride) + hd) * elt, cache_bytes(dt, L, planes, H, cols, D),
                         paged ? b4 * max_pages : 0, paged ? 0u : 4u, b4, b4 + 4};
  const void *outs[] = {out, lse, status};
  const size_t out_n[] = {T * hd * elt, static_cast<size_t>(T) * H * G * 4, b4};
  for (int o = 0; o < 3; ++o) {
    for (int j = 0; j < 6; ++j)
      if (overlaps(outs[o], out_n[o], ins[j], in_n[j])) return SPEC_EINVAL;
    for (int j = o + 1; j < 3; ++j)
      if (overlaps(outs[o], out_n[o], outs[j], out_n[j])) return SPEC_EINVAL;
  }
  P.T = T;
  P.cu = cu;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  if (dt == SPEC_BF16)
    return D <= 64 ? launch_prompt<__bf16, 64>(P, s)
                   : D <= 128 ? launch_prompt<__bf16, 128>(P, s) : launch_prompt<__bf16, 256>(P, s);
  return D <= 64 ? launch_prompt<float, 64>(P, s)
                 : D <= 128 ? launch_prompt<float, 128>(P, s) : launch_prompt<float, 256>(P, s);
}

}  // namespace
}  // namespace specv

using namespace specv;

extern "C" int spec_prompt_attention(const void *q, int64_t q_stride, const void *kv, spec_dtype dt, int L, int B,
                                     int H, int C, int D, int layer, int T, int G, const int32_t *end_col,
                                     const int32_t *kv_len, const int32_t *cu_seqlens, float scale, void *out,
                                     float *lse, int32_t *status, spec_stream_t stream) {
  return prompt_call(q, q_stride, kv, dt, L, B, B, H, C, D, layer, T, G, nullptr, 0, false, end_col, kv_len,
                     cu_seqlens, scale, out, lse, status, stream);
}

extern "C" int spec_prompt_attention_paged(const void *q, int64_t q_stride, const void *pool, spec_dtype dt, int L,
                                           int pages, int H, int page_size, int D, int layer, int B, int T, int G,
                                           const int32_t *block_table, int max_pages, const int32_t *kv_len,
                                           const int32_t *cu_seqlens, float scale, void *out, float *lse,
                                           int32_t *status, spec_stream_t stream) {
  return prompt_call(q, q_stride, pool, dt, L, pages, B, H, page_size, D, layer, T, G, block_table, max_pages, true,
                     nullptr, kv_len, cu_seqlens, scale, out, lse, status, stream);
}
