// How decode attention over the eight-bit cache shares its work: the blocks of all (sequence,
// kv head) pairs in a row, cut into equal pieces, one for each CTA.
//
// Lengths are on the device, so a warp of each CTA makes the plan (two lengths a lane and a
// scan).  A piece may begin and end within a pair: what a CTA finds there is a
// part, (O, m, l) in the scratch, and the join adds a pair's parts in the order of the
// CTAs.  A CTA has at most two of them, of its first pair and of its last; pairs that lie
// within a piece are finished where they are.
//
// A pair's beginning takes a CTA as long as some blocks do, and counts like them in the pieces'
// borders (ee_decode_pieces.cuh).  (Without that CTAs with several short pairs were done last: 18 us,
// where half of all were done in 14.)  Where all pairs can be cut by themselves into pieces that are
// no longer, no CTA has blocks of two, and beginnings do not count (8 sequences of 500, 8 kv heads:
// 10.9 us with the beginnings counted, 9.3 without).
#pragma once

#include <algorithm>
#include <type_traits>

#include "ee_cache_ops.cuh"
#include "ee_decode_pieces.cuh"
#include "ee_tcgen05.cuh"

namespace ee {

struct DecodePlan : DecodePieces {
  int tokens[2], base[2], size[2];  // of sequences lane and lane + 32: their places, and those before them
  int total, begin, end;

  // `least`: places of a piece at least.  whole: a CTA takes the pairs that begin in its
  // piece.  The whole warp.
  EE_DEV void init(const DecodeParams& p, int pieces, int least, bool whole, int me) {
    static_assert(EE_MAX_BATCH <= 64, "two sequences per lane");
    const int lane = threadIdx.x & 31;
    int at[2];  // both loads before either is waited for
#pragma unroll
    for (int u = 0; u < 2; ++u) at[u] = lane + 32 * u < p.batch ? p.pos[lane + 32 * u] : -1;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      tokens[u] = checked_length(at[u] == INT32_MAX ? at[u] : at[u] + 1, p.c.max_ctx, p.c.err);
      size[u] = (tokens[u] + 15) >> 4;
    }
    const int blocks = (int)__reduce_add_sync(0xffffffffu, size[0] + size[1]);
    const int pairs = __popc(__ballot_sync(0xffffffffu, size[0] > 0)) + __popc(__ballot_sync(0xffffffffu, size[1] > 0));
    cut(p.c.n_kv_heads, blocks, pairs, pieces, least);
    if (!whole) {
#pragma unroll
      for (int c = 8; c <= 32; c += 8)
        cut_alone(c, (int)__reduce_add_sync(0xffffffffu, (size[0] + c - 1) / c + (size[1] + c - 1) / c), pieces);
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) size[u] = places(size[u]);
    // both scans at once: sums of 32 sequences' places are below 2^16
    static_assert((32 + kCacheMaxCtx / 16) * 32 < 1 << 16, "two sums in a word");
    const uint32_t mine = (uint32_t)size[0] | (uint32_t)size[1] << 16;
    uint32_t sum = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t x = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += x;
    }
    const uint32_t all = __shfl_sync(0xffffffffu, sum, 31);
    sum -= mine;
    base[0] = (int)(sum & 0xffffu);
    base[1] = (int)(all & 0xffffu) + (int)(sum >> 16);
    total = ((int)(all & 0xffffu) + (int)(all >> 16)) * hkv;
    begin = min(total, me * each);
    end = min(total, begin + each);
    if (whole) {
      begin = next_pair(begin);
      end = next_pair(end);
    }
  }
  // The lane's sequence u holds place c.
  EE_DEV bool holds(int u, int c) const { return c >= base[u] * hkv && c < (base[u] + size[u]) * hkv; }
  // Value a[u] of the sequence that holds place c < total.
  EE_DEV int of(const int (&a)[2], unsigned lo, unsigned hi) const {
    return lo ? __shfl_sync(0xffffffffu, a[0], __ffs(lo) - 1) : __shfl_sync(0xffffffffu, a[1], __ffs(hi) - 1);
  }
  EE_DEV int next_pair(int c) const {  // the first pair that begins at c or behind it
    if (c >= total) return total;
    const unsigned lo = __ballot_sync(0xffffffffu, holds(0, c)), hi = __ballot_sync(0xffffffffu, holds(1, c));
    const int len = of(size, lo, hi), b0 = of(base, lo, hi) * hkv;
    return b0 + (c - b0 + len - 1) / len * len;
  }
  // The share of CTA `me` of the pair that holds place *c, or of the next one that has any (s = -1:
  // no more); *c: behind the pair.
  EE_DEV Share at(int* c, int me) const {
    Share r;
    for (;;) {
      r.s = -1;
      r.blocks = 0;
      if (*c >= end) return r;
      const unsigned lo = __ballot_sync(0xffffffffu, holds(0, *c)), hi = __ballot_sync(0xffffffffu, holds(1, *c));
      const int s = lo ? __ffs(lo) - 1 : 31 + __ffs(hi), b0 = of(base, lo, hi) * hkv, n = of(tokens, lo, hi);
      if (share(c, me, begin, end, s, b0, n, &r)) return r;
    }
  }
};

// Units or shares on their way from the warp that finds (and loads) them to those that work on
// them: code that stands once in the kernel, because a CTA's first instructions take as
// long to come as its first tiles.
template <typename T>
struct Ring {
  static constexpr int kDepth = 4;
  uint64_t full[kDepth], free[kDepth];
  T at[kDepth];

  EE_DEV void init(int readers) {  // one lane per place
    const int lane = threadIdx.x & 31;
    if (lane < kDepth) {
      mbar_init(&full[lane], 1);
      mbar_init(&free[lane], readers);
    }
  }
  EE_DEV bool put(int i, const T& x, int32_t* err) {
    if (i >= kDepth && !warp_wait(&free[i % kDepth], (i / kDepth - 1) & 1, err, DERR_EMPTY_WAIT)) return false;
    if ((threadIdx.x & 31) == 0) {
      at[i % kDepth] = x;
      mbar_arrive(&full[i % kDepth]);
    }
    __syncwarp();
    return true;
  }
  EE_DEV bool get(int i, T* x, int32_t* err) {
    if (!warp_wait(&full[i % kDepth], (i / kDepth) & 1, err, DERR_FULL_WAIT)) return false;
    *x = at[i % kDepth];
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&free[i % kDepth]);
    return true;
  }
};

// A join: a CTA adds the parts of J query heads of a sequence: 8 / J warps each, kAtOnce parts in
// flight a warp.  J is as small as two CTAs per SM allow: CTAs start 6 ns after one another,
// whatever they do (one for each of 4096 rows took 20 us), but a warp that walks many parts takes
// long too (one sequence of 16384 tokens, 57 parts: 13 us, with J = G = 4 17).
constexpr int kJoinThreads = 256;

template <int HD, int J>
struct Join {
  static constexpr int P = HD / 32, kAtOnce = 8, kStripes = 8 / J;  // a lane's dims; parts; warps of a head
  struct Stripes {
    float m[8], l[8], o[8][HD];
  };
  float m = -INFINITY, l = 0.0f, o[P] = {};

  // (m, l, O) of parts; m = -inf and l = 0: nothing was seen, and O is 0.  A factor may go to 0, but
  // every part is multiplied: an infinity or NaN of l and O stays.  (A part of NaN alone has no
  // maximum.)
  EE_DEV void add(const float (&mk)[kAtOnce], const float (&lk)[kAtOnce], const float (&x)[kAtOnce][P]) {
    float mn = m;
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) mn = fmaxf(mn, mk[u]);
    const float a = m == mn ? 1.0f : ex2(m - mn);
    m = mn;
    l *= a;
#pragma unroll
    for (int i = 0; i < P; ++i) o[i] *= a;
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      const float f = mk[u] == m ? 1.0f : ex2(mk[u] - m);
      l = fmaf(f, lk[u], l);
#pragma unroll
      for (int i = 0; i < P; ++i) o[i] = fmaf(f, x[u][i], o[i]);
    }
  }
  // All warps' sums, written to J heads side by side: 0 where nothing was seen.
  EE_DEV void finish(Stripes& all, uint16_t* to) const {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (lane == 0) {
      all.m[warp] = m;
      all.l[warp] = l;
    }
#pragma unroll
    for (int i = 0; i < P; ++i) all.o[warp][lane * P + i] = o[i];
    __syncthreads();
    for (int i = tid; i < J * HD; i += kJoinThreads) {
      const int head = i / HD, d = i % HD;
      float mm = -INFINITY, sum = 0.0f, y = 0.0f;
#pragma unroll
      for (int w = 0; w < kStripes; ++w) mm = fmaxf(mm, all.m[w * J + head]);
#pragma unroll
      for (int w = 0; w < kStripes; ++w) {
        const int at = w * J + head;
        const float f = all.m[at] == mm ? 1.0f : ex2(all.m[at] - mm);
        sum = fmaf(f, all.l[at], sum);
        y = fmaf(f, all.o[at][d], y);
      }
      const float il = sum > 0.0f ? 1.0f / sum : (sum == 0.0f ? 0.0f : sum);  // NaN stays
      to[i] = float_to_half_bits(within_half(y * il));
    }
  }
};

// launch(J) with the J for this many rows, J as a type's value.
template <int G, typename Launch>
cudaError_t join_by_rows(int rows, int sms, Launch launch) {
  int J = 1;
  while (J < G && rows > 2 * sms * J) J *= 2;
  if constexpr (G >= 8)
    if (J == 8) return launch(std::integral_constant<int, 8>());
  if constexpr (G >= 4)
    if (J == 4) return launch(std::integral_constant<int, 4>());
  if constexpr (G >= 2)
    if (J == 2) return launch(std::integral_constant<int, 2>());
  return launch(std::integral_constant<int, 1>());
}

// Launches a join behind the kernel that writes the parts.  Its CTAs start where that one's end, and
// the first SMs to be free would take them all, eight or more each: shared memory that they do not
// use keeps them apart, as many on an SM as it takes, but no more of it than a CTA before them had.
// (16 sequences behind 1000 shared tokens: 15.1 -> 13.4 us, 8 behind 15000: 27.7 -> 26.0.)
template <typename... Params, typename... Args>
cudaError_t launch_join(void (*kernel)(Params...), int ctas, int sms, size_t before, cudaStream_t st, Args... args) {
  cudaFuncAttributes has;
  cudaError_t e = cudaFuncGetAttributes(&has, kernel);
  if (e != cudaSuccess) return e;
  const size_t per = (size_t)(ctas + sms - 1) / sms, taken = has.sharedSizeBytes + 1024, most = std::min<size_t>(before, 228 * 1024 / per);
  const size_t apart = most > taken ? (most - taken) & ~(size_t)1023 : 0;
  if (apart > (size_t)has.maxDynamicSharedSizeBytes) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)(227 * 1024 - has.sharedSizeBytes));
    if (e != cudaSuccess) return e;
  }
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(kJoinThreads);
  cfg.dynamicSmemBytes = apart;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace ee
