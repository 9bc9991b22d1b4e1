// Causal attention of packed prompt rows over the paged cache, on the tensor
// cores (tcgen05.mma, fp32 accumulators in tensor memory).
//
// A CTA owns 256 rows of S = Q K^T for one kv head: row r is query head r % G of
// the group at the prompt's position i0 + r / G, so that one read of K and V
// serves the whole group.  The rows are two M = 128 tiles with a softmax
// warpgroup each; while one is busy with its probabilities the tensor core works
// for the other:
//   warp 9 (one thread)  S_t = Q_t K_j^T, then O_t += P_t V_j, for t = 0, 1 in turn
//   warps 4t .. 4t + 3   a thread per row: S_t to registers, the running maximum
//                        and sum, P_t = exp2(c S - c m) as fp16 over S_t's columns
//   warp 8               K and V tiles of 128 keys by TMA, one copy per 16-slot
//                        block and 64 columns, into a ring of NST tiles
// The running maximum may lag behind by up to 8 (in log2): then P is at most 2^8
// instead of 1, which fp16 holds as exactly, and O, in tensor memory, is
// rescaled only when a row's maximum has grown by more than that.  The sum is
// kept in fp32 from the unrounded P; rounding P to fp16 (2^-11 of it) is the
// price of feeding the second product to the tensor core, and o is fp16 itself.
//
// Tiles that some row does not see whole are masked by comparing positions, so
// a NaN score is dropped as any other.  A NaN or infinity in V times a zero
// probability would not be: in those tiles the warpgroups replace such values by
// zero in shared memory, and where they stand for tokens of the sequence the
// rows that see them get them added at the end.
//
// Few rows over many keys (a chunk behind a long prefix): the keys are split over
// the CTAs of a cluster, which join their (O, m, l) through distributed shared
// memory in rank order.  No scratch, no atomics.
#include <cooperative_groups.h>
#include <math.h>

#include <atomic>

#include "ee_cache_ops.cuh"
#include "ee_tcgen05.cuh"

namespace cg = cooperative_groups;

namespace ee {
namespace {

constexpr int kRows = 256;     // rows of S per CTA: two tiles of 128
constexpr int kKeys = 128;     // keys per step
constexpr int kThreads = 320;  // two softmax warpgroups, TMA, MMA
constexpr int kMaxCluster = 8;

template <int HD>
struct Shape {
  static constexpr int H = HD / 64;                       // 64-column halves
  static constexpr uint32_t kTile = 128 * HD * 2;         // a Q, K or V tile
  static constexpr uint32_t kHalf = 128 * 128;            // one 64-column half of it
  static constexpr int NST = HD == 128 ? 4 : 6;           // ring tiles
  static constexpr size_t kSmem = 1024 + (2 + NST) * (size_t)kTile;
  static constexpr int kPad = HD + 4;                     // floats per joined row
  static_assert((size_t)kRows * kPad * 4 <= (2 + NST) * (size_t)kTile, "the join reuses the tiles' space");
};

struct Maps {
  CUtensorMap q, k, v;
};

struct Shared {
  uint64_t q_full, kv_full[8], kv_empty[8], s_full[2], p_ready[2], o_done[2];
  uint32_t tmem;
  int bad_v;            // a non-finite V value was replaced
  float m[kRows], l[kRows];
};

// log of the sum of exp(s / sqrt(hd)), from its sum l relative to the score m.
EE_DEV float log_sum(float m, float l, const Exponent& ex) {
  return l == 0.0f ? -INFINITY : fmaf(m, ex.unit_hi, fmaf(m, ex.unit_lo, logf(l)));
}

template <int HD, int G, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
    k_prompt_attention(const PromptParams p, const __grid_constant__ Maps maps, const Exponent ex) {
  using S = Shape<HD>;
  constexpr int kPos = kRows / G;  // positions per CTA
  const float c = ex.c;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Shared sh;
  uint8_t* tiles = reinterpret_cast<uint8_t*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int nsplit = SPLIT ? (int)cg::this_cluster().num_blocks() : 1;
  const int split = SPLIT ? (int)cg::this_cluster().block_rank() : 0;
  const int unit = blockIdx.x / nsplit;
  const int g = unit % p.c.n_kv_heads;
  const PromptTile tl = prompt_tile(p, unit / p.c.n_kv_heads, kPos);
  if (tl.s < 0) return;  // the whole cluster
  const int off = tl.sq.ctx - tl.sq.n;  // position of row 0

  // keys that tile t's rows see, in tiles: [0, nt[t]); those from jm[t] on are
  // not seen whole by every row
  int ka = 0, kb, nt[2], jm[2];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int r0 = tl.i0 + t * (kPos / 2), r1 = min(tl.sq.n, r0 + kPos / 2);
    nt[t] = r1 > r0 ? max(0, off + r1 + kKeys - 1) / kKeys : 0;
    jm[t] = max(0, off + r0 + 1) / kKeys;
  }
  kb = max(nt[0], nt[1]);
  if (SPLIT) {
    const int each = (kb + nsplit - 1) / nsplit;
    ka = min(kb, split * each);
    kb = min(kb, ka + each);
  }
  const int n0 = max(0, min(nt[0], kb) - ka), n1 = max(0, min(nt[1], kb) - ka), nk = kb - ka;

  if (tid == 0) {
    mbar_init(&sh.q_full, 1);
    for (int i = 0; i < S::NST; ++i) {
      mbar_init(&sh.kv_full[i], 1);
      mbar_init(&sh.kv_empty[i], 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&sh.s_full[t], 1);
      mbar_init(&sh.p_ready[t], 128);
      mbar_init(&sh.o_done[t], 1);
    }
    sh.bad_v = 0;
    fence_mbar_init();
  }
  if (warp == 9) tmem_alloc(&sh.tmem, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  const uint32_t q_s = smem_addr(tiles), kv_s = q_s + 2 * S::kTile;
  // tensor memory: S_t (128 columns, P_t over its first 64), then O_t
  auto s_col = [&](int t) { return tmem + t * 128; };
  auto o_col = [&](int t) { return tmem + 256 + t * HD; };

  if (warp == 8) {
    // ring item 2 j is K of key tile ka + j, item 2 j + 1 its V
    const int ntok = tl.sq.ctx, nblk = (ntok + 15) >> 4;
    const int32_t* bt = p.c.table + (int64_t)tl.s * p.c.table_stride;
    if (lane == 0 && nk > 0) {
      mbar_arrive_expect_tx(&sh.q_full, (n0 > 0 ? S::kTile : 0) + (n1 > 0 ? S::kTile : 0));
      for (int t = 0; t < 2; ++t)
        if ((t ? n1 : n0) > 0)
          for (int h = 0; h < S::H; ++h)
            tma_load_3d(q_s + t * S::kTile + h * S::kHalf, &maps.q, h * 64, g * G,
                        tl.sq.first + tl.i0 + t * (kPos / 2), &sh.q_full);
    }
    const int b8 = lane & 7, half = lane >> 3;
    auto block_id = [&](int j) {  // of block b8 of key tile j
      const int b = j * 8 + b8;
      int id = b < nblk && j < kb ? bt[b] : 0;
      if (id < 0 || id >= p.c.n_blocks) {
        report(p.c.err, EE_DERR_BLOCK);
        id = 0;
      }
      return id;
    };
    int id = block_id(ka), issued = 0;
    bool ok = true;
    for (int j = ka; j < kb && ok; ++j) {
      const int next = block_id(j + 1), here = min(8, nblk - j * 8);
      for (int kv = 0; kv < 2; ++kv, ++issued) {
        const int st = issued % S::NST, pass = issued / S::NST;
        if (pass > 0)
          ok = warp_wait(&sh.kv_empty[st], (pass - 1) & 1, p.c.err, DERR_EMPTY_WAIT);
        if (!ok) break;
        if (lane == 0) mbar_arrive_expect_tx(&sh.kv_full[st], (uint32_t)here * 16 * HD * 2);
        __syncwarp();
        if (half < S::H && b8 < here)
          tma_load_2d(kv_s + st * S::kTile + half * S::kHalf + b8 * 2048, kv ? &maps.v : &maps.k, half * 64,
                      (id * p.c.n_kv_heads + g) * 16, &sh.kv_full[st]);
      }
      id = next;
    }
    if (!ok)  // copies land before the CTA ends
      for (int i = max(0, issued - S::NST); i < issued; ++i)
        mbar_wait_bounded(&sh.kv_full[i % S::NST], (i / S::NST) & 1, p.c.err, DERR_DRAIN_WAIT);
  } else if (warp == 9) {
    if (lane == 0 && nk > 0) {
      constexpr uint32_t id_qk = instr_desc(0, kKeys, 128), id_pv = instr_desc(0, HD, 128, true);
      auto item = [&](int i) { return kv_s + (i % S::NST) * S::kTile; };
      auto landed = [&](int i) {
        const bool r = mbar_wait_bounded(&sh.kv_full[i % S::NST], (i / S::NST) & 1, p.c.err, DERR_FULL_WAIT);
        tc_fence_after();
        return r;
      };
      auto qk = [&](int t, int j) {
        const uint32_t a = q_s + t * S::kTile, b = item(2 * j);
#pragma unroll
        for (int kk = 0; kk < HD / 16; ++kk) {
          const uint32_t o = (kk >> 2) * S::kHalf + (kk & 3) * 32;
          mma_f16(s_col(t), smem_desc_sw128(a + o), smem_desc_sw128(b + o), id_qk, kk > 0);
        }
        mma_commit(&sh.s_full[t]);
      };
      auto pv = [&](int t, int j) {
        const uint32_t b = item(2 * j + 1);
#pragma unroll
        for (int kk = 0; kk < kKeys / 16; ++kk)
          mma_f16_ta(o_col(t), s_col(t) + kk * 8, smem_desc_sw128_mn(b + kk * 2048, S::kHalf), id_pv, j > 0 || kk > 0);
        mma_commit(&sh.o_done[t]);
      };
      bool ok = mbar_wait_bounded(&sh.q_full, 0, p.c.err, DERR_FULL_WAIT) && landed(0);
      if (ok) {
        if (n0 > 0) qk(0, 0);
        if (n1 > 0) qk(1, 0);
        mma_commit(&sh.kv_empty[0]);
      }
      for (int j = 0; j < nk && ok; ++j) {
        ok = landed(2 * j + 1);
        for (int t = 0; t < 2 && ok; ++t) {
          const int n = t ? n1 : n0;
          if (j < n) {
            ok = mbar_wait_bounded(&sh.p_ready[t], j & 1, p.c.err, DERR_FULL_WAIT);
            tc_fence_after();
            if (ok) pv(t, j);
          }
          if (t == 1) mma_commit(&sh.kv_empty[(2 * j + 1) % S::NST]);
          if (t == 0 && j + 1 < nk && ok) ok = landed(2 * j + 2);
          if (j + 1 < n && ok) qk(t, j + 1);
          if (t == 1 && j + 1 < nk) mma_commit(&sh.kv_empty[(2 * j + 2) % S::NST]);
        }
      }
    }
    __syncwarp();
  } else {
    const int t = warp >> 2, r = tid & 127;  // tile and row
    const int n = t ? n1 : n0;
    const int row = tl.i0 + t * (kPos / 2) + r / G;
    const bool valid = row < tl.sq.n;
    const int pos = valid ? off + row : -1;  // last key this row sees
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_at = s_col(t) + lane_base, o_at = o_col(t) + lane_base;
    float m = -INFINITY, l = 0.0f;
    bool ok = true;
    for (int j = 0; j < n; ++j) {
      if (!(ok = warp_wait(&sh.s_full[t], j & 1, p.c.err, DERR_FULL_WAIT))) break;
      tc_fence_after();
      uint32_t s[kKeys];
#pragma unroll
      for (int i = 0; i < 4; ++i) tmem_ld32(s_at + 32 * i, s + 32 * i);
      tmem_wait_ld();
      tmem_pin<kKeys>(s);
      const bool masked = ka + j >= jm[t];
      if (masked) {
        const int lim = pos - (ka + j) * kKeys;
#pragma unroll
        for (int i = 0; i < kKeys; ++i)
          if (i > lim) s[i] = 0xff800000u;  // -inf
      }
      float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int i = 0; i < kKeys; i += 8)
#pragma unroll
        for (int u = 0; u < 4; ++u)
          mx[u] = fmaxf(mx[u], fmaxf(__uint_as_float(s[i + u]), __uint_as_float(s[i + 4 + u])));
      const float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
      if (j == 0) {
        m = mt;
      } else if (__any_sync(0xffffffffu, (mt - m) * c > 8.0f)) {
        // some row's maximum has grown too far: this warp's rows of O and l go
        // over to the new maxima, once the product before has been added
        const float mn = fmaxf(m, mt);
        const float a = m == mn ? 1.0f : ex2((m - mn) * c);
        m = mn;
        l *= a;
        if (!(ok = warp_wait(&sh.o_done[t], (j - 1) & 1, p.c.err, DERR_FULL_WAIT))) break;
        tc_fence_after();
#pragma unroll 1
        for (int i = 0; i < HD; i += 16) {
          uint32_t o[16];
          tmem_ld16(o_at + i, o);
          tmem_wait_ld();
          tmem_pin<16>(o);
#pragma unroll
          for (int u = 0; u < 16; ++u) o[u] = __float_as_uint(__uint_as_float(o[u]) * a);
          tmem_st16(o_at + i, o);
        }
      }
      // a row that has seen nothing yet has m = -inf: its P is 0
      const float mc = m == -INFINITY ? 0.0f : m * c;
      const uint64_t c2 = pack2(c, c), nm2 = pack2(-mc, -mc);
      uint64_t sum[2] = {0, 0};
#pragma unroll
      for (int i = 0; i < kKeys; i += 32) {
        uint32_t ph[16];
#pragma unroll
        for (int u = 0; u < 32; u += 2) {
          const float2 x =
              unpack2(fma2(pack2(__uint_as_float(s[i + u]), __uint_as_float(s[i + u + 1])), c2, nm2));
          const float e0 = ex2(x.x), e1 = ex2(x.y);
          sum[(u >> 1) & 1] = add2(sum[(u >> 1) & 1], pack2(e0, e1));
          const __half2 h = __floats2half2_rn(e0, e1);
          ph[u >> 1] = *reinterpret_cast<const uint32_t*>(&h);
        }
        tmem_st16(s_at + i / 2, ph);
      }
      const float2 st = unpack2(add2(sum[0], sum[1]));
      l += st.x + st.y;
      if (masked) {
        // V values that are not finite become 0 before the product reads them
        const int it = 2 * j + 1;
        if (!(ok = warp_wait(&sh.kv_full[it % S::NST], (it / S::NST) & 1, p.c.err, DERR_FULL_WAIT))) break;
        uint8_t* vt = tiles + 2 * S::kTile + (it % S::NST) * S::kTile;
        bool fixed = false;
#pragma unroll 4
        for (int i = r; i < (int)(S::kTile / 16); i += 128) {
          uint4 v = *reinterpret_cast<uint4*>(vt + i * 16);
          uint32_t* w = reinterpret_cast<uint32_t*>(&v);
          bool any = false;
#pragma unroll
          for (int u = 0; u < 4; ++u) any |= ((w[u] & 0x7c007c00u) + 0x04000400u) & 0x80008000u;
          if (any) {
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              if ((w[u] & 0x7c00u) == 0x7c00u) w[u] &= 0xffff0000u;
              if ((w[u] & 0x7c000000u) == 0x7c000000u) w[u] &= 0x0000ffffu;
            }
            *reinterpret_cast<uint4*>(vt + i * 16) = v;
            // rows of the tile are 128 bytes in each half
            if ((ka + j) * kKeys + (int)((i * 16) % S::kHalf) / 128 < tl.sq.ctx) fixed = true;
          }
        }
        if (fixed) sh.bad_v = 1;
        fence_proxy_async();
      }
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(&sh.p_ready[t]);
    }
    if (ok && n > 0) ok = warp_wait(&sh.o_done[t], (n - 1) & 1, p.c.err, DERR_FULL_WAIT);
    tc_fence_after();
    asm volatile("bar.sync 1, 256;" ::: "memory");  // bad_v of both tiles; the tiles' space is free
    const bool bad = sh.bad_v;
    const int head = g * G + r % G;
    const float il = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);  // NaN stays
    uint16_t* orow = p.o + (int64_t)(tl.sq.first + row) * p.o_stride + head * HD;
    float* jrow = reinterpret_cast<float*>(tiles) + (size_t)(t * 128 + r) * S::kPad;
#pragma unroll 1
    for (int i = 0; i < HD; i += 32) {
      uint32_t o[32];
      tmem_ld32(o_at + i, o);
      tmem_wait_ld();
      tmem_pin<32>(o);
      if (n == 0) {
#pragma unroll
        for (int u = 0; u < 32; ++u) o[u] = 0;
      }
      if (bad) {  // the values taken out above, for the rows that see them
        const int end = min(pos, kb * kKeys - 1);
        for (int tok = max(min(jm[0], jm[1]), ka) * kKeys; tok <= end; ++tok) {
          bool bok;
          const int b = checked_block(p.c.table, p.c.table_stride, p.c.n_blocks, tl.s, tok, nullptr, &bok);
          const uint16_t* v = p.c.v + (((size_t)b * p.c.n_kv_heads + g) * 16 + (tok & 15)) * HD + i;
#pragma unroll
          for (int u = 0; u < 32; ++u)
            if ((v[u] & 0x7c00u) == 0x7c00u)
              o[u] = __float_as_uint(__uint_as_float(o[u]) + __half2float(__ushort_as_half(v[u])));
        }
      }
      if (SPLIT) {
#pragma unroll
        for (int u = 0; u < 32; u += 4)
          *reinterpret_cast<uint4*>(jrow + i + u) = make_uint4(o[u], o[u + 1], o[u + 2], o[u + 3]);
      } else if (valid) {
#pragma unroll
        for (int u = 0; u < 32; u += 8) {
          uint32_t h[4];
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const __half2 x = __floats2half2_rn(__uint_as_float(o[u + 2 * w]) * il, __uint_as_float(o[u + 2 * w + 1]) * il);
            h[w] = *reinterpret_cast<const uint32_t*>(&x);
          }
          *reinterpret_cast<uint4*>(orow + i + u) = make_uint4(h[0], h[1], h[2], h[3]);
        }
      }
    }
    if (SPLIT) {
      sh.m[t * 128 + r] = m;
      sh.l[t * 128 + r] = l;
    } else if (valid && p.lse) {
      p.lse[(size_t)head * p.total_q + tl.sq.first + row] = log_sum(m, l, ex);
    }
    tc_fence_before();
  }
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_free(tmem, 512);
  }
  if (SPLIT) {
    // rank r joins rows r, r + nsplit, ...: every rank's (O, m, l) in rank order
    cg::cluster_group cl = cg::this_cluster();
    cl.sync();
    constexpr int L = HD / 4;  // threads per row
    const int rows = min(kRows, (tl.sq.n - tl.i0) * G);
    if (tid < 256) {
      for (int r = split + nsplit * (tid / L); r < rows; r += nsplit * (256 / L)) {
        const int row = tl.i0 + r / G, head = g * G + r % G, col = (tid % L) * 4;
        float M = -INFINITY;
        float mr[kMaxCluster], lr[kMaxCluster];
        float4 x[kMaxCluster];
#pragma unroll
        for (int k = 0; k < kMaxCluster; ++k) {
          if (k >= nsplit) break;
          const Shared* o = cl.map_shared_rank(&sh, k);
          mr[k] = o->m[r];
          lr[k] = o->l[r];
          x[k] = *reinterpret_cast<const float4*>(cl.map_shared_rank(reinterpret_cast<float*>(tiles), k) +
                                                  (size_t)r * S::kPad + col);
          M = fmaxf(M, mr[k]);
        }
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        float l = 0.0f;
#pragma unroll
        for (int k = 0; k < kMaxCluster; ++k) {
          if (k >= nsplit) break;
          if (lr[k] == 0.0f) continue;  // saw nothing (NaN is not 0)
          const float a = mr[k] == M ? 1.0f : ex2((mr[k] - M) * c);
          l += a * lr[k];
          o.x += a * x[k].x;
          o.y += a * x[k].y;
          o.z += a * x[k].z;
          o.w += a * x[k].w;
        }
        const float il = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);
        const __half2 h0 = __floats2half2_rn(o.x * il, o.y * il), h1 = __floats2half2_rn(o.z * il, o.w * il);
        *reinterpret_cast<uint2*>(p.o + (int64_t)(tl.sq.first + row) * p.o_stride + head * HD + col) =
            make_uint2(*reinterpret_cast<const uint32_t*>(&h0), *reinterpret_cast<const uint32_t*>(&h1));
        if (col == 0 && p.lse)
          p.lse[(size_t)head * p.total_q + tl.sq.first + row] = log_sum(M, l, ex);
      }
    }
    cl.sync();  // nobody leaves while its memory is read
  }
}

template <int HD, int G>
cudaError_t launch_t(const PromptParams& p, cudaStream_t st) {
  using S = Shape<HD>;
  static std::atomic<uint64_t> prepared{0};  // a bit per device
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !(prepared.load(std::memory_order_acquire) >> dev & 1)) {
    e = cudaFuncSetAttribute(k_prompt_attention<HD, G, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(k_prompt_attention<HD, G, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
    if (e != cudaSuccess) return e;
    if (dev < 64) prepared.fetch_or(1ull << dev, std::memory_order_release);
  }
  e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  Maps maps;
  const uint64_t qd[3] = {(uint64_t)HD, (uint64_t)p.n_heads, (uint64_t)p.total_q};
  const uint64_t qs[2] = {(uint64_t)HD * 2, (uint64_t)p.q_stride * 2};
  const uint32_t qb[3] = {64, (uint32_t)G, 128 / (uint32_t)G};
  const uint64_t cd[2] = {(uint64_t)HD, (uint64_t)p.c.n_blocks * p.c.n_kv_heads * 16}, cs[1] = {(uint64_t)HD * 2};
  const uint32_t cb[2] = {64, 16};
  if (!encode_tensor_map(&maps.q, false, 3, p.q, qd, qs, qb) || !encode_tensor_map(&maps.k, false, 2, p.c.k, cd, cs, cb) ||
      !encode_tensor_map(&maps.v, false, 2, p.c.v, cd, cs, cb))
    return cudaErrorInvalidValue;
  const Exponent ex = make_exponent(HD);
  // at most this many tiles: each sequence may leave one unfilled
  const int64_t units = ((int64_t)p.total_q * G / kRows + p.n_seqs) * p.c.n_kv_heads;
  int split = 1;
  while (split < kMaxCluster && units * split * 2 <= sms && split * 2 * kKeys < p.c.max_ctx) split *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(units * split));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = S::kSmem;
  cfg.stream = st;
  if (split == 1) return cudaLaunchKernelEx(&cfg, k_prompt_attention<HD, G, false>, p, maps, ex);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = split;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_prompt_attention<HD, G, true>, p, maps, ex);
}

}  // namespace

cudaError_t launch_prompt_attention(const PromptParams& p, cudaStream_t st) {
  const int G = p.n_heads / p.c.n_kv_heads, hd = p.c.head_dim;
#define EE_PROMPT_CASE(HD_, G_) \
  if (hd == HD_ && G == G_) return launch_t<HD_, G_>(p, st);
  EE_PROMPT_CASE(64, 1)
  EE_PROMPT_CASE(64, 2)
  EE_PROMPT_CASE(64, 4)
  EE_PROMPT_CASE(64, 8)
  EE_PROMPT_CASE(128, 1)
  EE_PROMPT_CASE(128, 2)
  EE_PROMPT_CASE(128, 4)
  EE_PROMPT_CASE(128, 8)
#undef EE_PROMPT_CASE
  return cudaErrorInvalidValue;
}

}  // namespace ee
