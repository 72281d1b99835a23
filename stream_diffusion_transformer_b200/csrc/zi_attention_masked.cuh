// Attention with capped scores, a distance bias and masks (head_dim 128, bf16 in and out,
// fp32 scores and softmax):
//   s_ij = scale q_i . k_j;  s = cap tanh(s / cap) (cap > 0);  s -= slope_h |p_i - j|;
//   o_i = sum_j softmax_j(s_ij) v_j over the keys j that query i sees, 0 if it sees none,
// where element b has n_b keys, its queries are the last of them (p_i = i + n_b - q_len),
// and i sees j when j < n_b, and (causal) j <= p_i or j < prefix_b, and (documents) their
// ids are equal and not negative.
#pragma once
#include "zi_attention.cuh"
#include "zi_cluster.cuh"
#include "zi_common.cuh"

namespace zi {

struct MaskedParams {
  const uint16_t *q, *k, *v;
  uint16_t* out;
  long long q_bs, q_rs, q_hs, k_bs, k_rs, k_hs, v_bs, v_rs, v_hs, o_bs, o_rs, o_hs;  // strides in elements
  int batch, heads, kv_heads, group, q_len, kv_len;
  float scale_log2;     // scale * log2(e); with a cap: scale / cap
  float cap_log2;       // cap * log2(e), 0 = no cap
  int cap_poly;         // the cap's polynomial can be used (its coefficients' powers of the scale stay in range)
  const float* slopes;  // [heads] or null
  int causal;
  const int* prefix;    // [batch] or null
  const int* lengths;   // [batch] or null
  const int *q_doc, *k_doc;  // [batch, q_len], [batch, kv_len], or null
  int head_group;            // key heads whose units run side by side (attention_many_kernel)
};

// Keys of element b.
ZI_DEV int masked_keys(const MaskedParams& p, int b) {
  if (!p.lengths) return p.kv_len;
  return max(0, min(p.kv_len, __ldg(p.lengths + b)));
}

// First key past those that query i of an element with n keys sees.
ZI_DEV int masked_limit(const MaskedParams& p, int b, int i, int n) {
  if (!p.causal) return n;
  const int upto = i + n - p.q_len + 1;
  const int pre = p.prefix ? __ldg(p.prefix + b) : 0;
  return max(0, min(n, max(upto, pre)));
}

ZI_DEV float fast_rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// tanh to a relative error of 10^-6 or less, so that scores far below their cap keep their own accuracy.  From 1/4 on
// 1 - 2 / (e^2x + 1), whose error is a few 2^-24 whatever the result's size (infinite e^2x gives 1, e^2x = 0 gives
// -1); below it the series up to x^7, whose next term is 62/2835 x^8 < 2^-21 of x.
ZI_DEV float tanh_score(float x) {
  const float u = x * x;
  const float low = x * fmaf(u, fmaf(u, fmaf(u, -17.f / 315.f, 2.f / 15.f), -1.f / 3.f), 1.f);
  const float high = 1.f - 2.f * fast_rcp(fast_exp2(x * 2.885390081777927f) + 1.f);
  return fabsf(x) < 0.25f ? low : high;
}

// ------------------------------------------------------------------ few queries
// One CTA per 16 rows of a key head (a row is one query of one head of the group, row =
// query * group + head in the group) and share of the keys; a cluster of CTAs shares a
// tile's keys.  Bound by reading K and V: each of the 4 warps streams its own chunks of 16
// keys through a private smem ring with TMA (3 chunks of K and V deep, 24 KB per warp, two
// CTAs per SM), takes scores and products with mma.sync m16n8k16 (16 rows padded: the tensor
// work is small beside the loads) and keeps its own running maximum and sum.  The warps' and
// then the cluster's partials are joined in a fixed order.  One query over 2 x 16,896 keys, 30 heads: 80.9 us,
// 5.6 TB/s.
namespace few {
constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kChunk = 16;                       // keys per chunk
constexpr int kRing = 3;
constexpr uint32_t kBox = kChunk * 128;          // 16 rows of 64 dims, 128-byte swizzle
constexpr uint32_t kChunkBytes = 4 * kBox;       // K dims 0..63, 64..127, then V
constexpr uint32_t kWarpBytes = kRing * kChunkBytes;
constexpr uint32_t kBar = kWarps * kWarpBytes;
constexpr uint32_t kSmemBytes = kBar + 256 + 1024;
constexpr uint32_t kPartFloats = 16 * 128 + 32;  // O [16][128], then m [16], l [16]
static_assert((kWarps + 1) * kPartFloats * 4 <= kBar, "partials reuse the ring");
}  // namespace few

ZI_DEV void tma_load_4d(void* smem_dst, const CUtensorMap* map, uint64_t* bar, int x, int y, int z, int w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], [%2];" ::
          "r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "r"(w)
      : "memory");
}

ZI_DEV void ldsm4(uint32_t* r, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
ZI_DEV void ldsm4_t(uint32_t* r, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
ZI_DEV void mma16816(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__global__ void __launch_bounds__(few::kThreads)
    attention_few_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, MaskedParams p,
                         int splits) {
  using namespace few;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kBar);  // [kWarps][kRing]
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + kWarps * kRing);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = int(blockIdx.x) % splits, tile = int(blockIdx.x) / splits;
  const int hk = blockIdx.y, b = blockIdx.z;
  const int rows = p.q_len * p.group;
  const int row0 = tile * 16;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kWarps * kRing; ++i) mbar_init(bars + i, 1);
    *abort_flag = device_error_set() ? 1 : 0;  // an earlier kernel timed out: leave everything untouched
    fence_mbar_init();
    prefetch_tmap(&tmK);
    prefetch_tmap(&tmV);
  }
  __syncthreads();

  const int n = masked_keys(p, b);
  // keys that any row of the tile may see: limits grow with the query
  const int i_last = (min(row0 + 16, rows) - 1) / p.group;
  const int end = *abort_flag ? 0 : masked_limit(p, b, i_last, n);
  const int chunks = (end + kChunk - 1) / kChunk;
  const int c0 = int(static_cast<long long>(rank) * chunks / splits) + warp;
  const int c1 = int(static_cast<long long>(rank + 1) * chunks / splits);
  uint8_t* ring = smem + warp * kWarpBytes;
  uint64_t* full = bars + warp * kRing;
  auto load = [&](int c, int slot) {  // lane 0
    uint8_t* dst = ring + slot * kChunkBytes;
    mbar_arrive_expect_tx(&full[slot], kChunkBytes);
    tma_load_4d(dst, &tmK, &full[slot], 0, hk, c * kChunk, b);
    tma_load_4d(dst + kBox, &tmK, &full[slot], 64, hk, c * kChunk, b);
    tma_load_4d(dst + 2 * kBox, &tmV, &full[slot], 0, hk, c * kChunk, b);
    tma_load_4d(dst + 3 * kBox, &tmV, &full[slot], 64, hk, c * kChunk, b);
  };
  if (lane == 0)
    for (int s = 0; s < kRing; ++s)
      if (c0 + s * kWarps < c1) load(c0 + s * kWarps, s);

  // this lane's two rows (fragment rows lane / 4 and lane / 4 + 8) and their Q fragments: 8 steps of 16 dims
  int lim[2], pos[2], doc[2];
  float slope[2];
  uint32_t qf[8][4];
  const int gid = lane >> 2, tid = lane & 3;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int r = row0 + gid + 8 * h;
    const int i = r / p.group, g = r - i * p.group;
    const bool have = r < rows;
    lim[h] = have ? masked_limit(p, b, i, n) : 0;
    pos[h] = i + n - p.q_len;
    doc[h] = have && p.q_doc ? __ldg(p.q_doc + size_t(b) * p.q_len + i) : 0;
    if (doc[h] < 0) lim[h] = 0;
    slope[h] = have && p.slopes ? __ldg(p.slopes + hk * p.group + g) * 1.4426950408889634f : 0.f;
    const uint16_t* src = p.q + b * p.q_bs + i * p.q_rs + (hk * p.group + g) * p.q_hs;
#pragma unroll
    for (int s = 0; s < 8; ++s) {
      qf[s][h] = have ? __ldg(reinterpret_cast<const uint32_t*>(src + s * 16 + tid * 2)) : 0u;
      qf[s][2 + h] = have ? __ldg(reinterpret_cast<const uint32_t*>(src + s * 16 + 8 + tid * 2)) : 0u;
    }
  }
  const int all_lim = __reduce_min_sync(0xffffffffu, min(row0 + gid < rows ? lim[0] : 0x7fffffff,
                                                         row0 + gid + 8 < rows ? lim[1] : 0x7fffffff));
  const int* kd = p.k_doc ? p.k_doc + size_t(b) * p.kv_len : nullptr;

  float o[16][4];
#pragma unroll
  for (int t = 0; t < 16; ++t) o[t][0] = o[t][1] = o[t][2] = o[t][3] = 0.f;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  const int lr = lane & 7, lm = lane >> 3;  // ldmatrix: this lane's row in matrix lm
  int slot = 0;
  uint32_t phase = 0;
  for (int c = c0; c < c1; c += kWarps) {
    // ids of the keys 2 tid, 2 tid + 1 and 8 further, as the fragments hold them
    int id[4] = {0, 0, 0, 0};
    const bool part = kd || (c + 1) * kChunk > all_lim;
    uint32_t used[2] = {~0u, ~0u};  // V rows that some query may see, as pairs of bf16
    if (part) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int key = c * kChunk + (e >> 1) * 8 + tid * 2 + (e & 1);
        if (kd) id[e] = key < n ? __ldg(kd + key) : -1;
        if (key >= n || id[e] < 0) used[e >> 1] &= (e & 1) ? 0x0000FFFFu : 0xFFFF0000u;
      }
    }
    if (!mbar_wait_warp(&full[slot], phase, abort_flag, ZI_DEVERR_TIMEOUT_SOFTMAX)) break;
    const uint32_t ks = smem_u32(ring + slot * kChunkBytes), vs = ks + 2 * kBox;
    float s[2][4];
#pragma unroll
    for (int t = 0; t < 2; ++t) s[t][0] = s[t][1] = s[t][2] = s[t][3] = 0.f;
#pragma unroll
    for (int kp = 0; kp < 4; ++kp) {  // two 16-dim steps at a time
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        uint32_t kf[4];
        ldsm4(kf, ks + (kp >> 1) * kBox + (t * 8 + lr) * 128 + ((((kp & 1) * 4 + lm) ^ lr) << 4));
        mma16816(s[t], qf[2 * kp], kf[0], kf[1]);
        mma16816(s[t], qf[2 * kp + 1], kf[2], kf[3]);
      }
    }
    // scores to the exp2 domain, masked
    float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int t = 0; t < 2; ++t) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int h = e >> 1, key = c * kChunk + t * 8 + tid * 2 + (e & 1);
        float y = s[t][e] * p.scale_log2;
        if (p.cap_log2 != 0.f) y = tanh_score(y) * p.cap_log2;
        if (p.slopes) y -= slope[h] * fabsf(float(pos[h] - key));
        if (part && (key >= lim[h] || (kd && id[t * 2 + (e & 1)] != doc[h]))) y = -INFINITY;
        s[t][e] = y;
        mx[h] = fmaxf(mx[h], y);
      }
    }
    float mu[2];
    bool grows = false;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 1));
      mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 2));
      grows = grows || mx[h] > m[h] + 8.f;  // the maximum may lag by 2^8
    }
    if (__any_sync(0xffffffffu, grows)) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (mx[h] > m[h] + 8.f) {  // each row by its own scores alone
          const float alpha = m[h] == -INFINITY ? 0.f : fast_exp2(m[h] - mx[h]);
          m[h] = mx[h];
          l[h] *= alpha;
#pragma unroll
          for (int t = 0; t < 16; ++t) {
            o[t][2 * h] *= alpha;
            o[t][2 * h + 1] *= alpha;
          }
        }
      }
    }
    mu[0] = m[0] == -INFINITY ? 0.f : m[0];  // a row that has seen nothing yet
    mu[1] = m[1] == -INFINITY ? 0.f : m[1];
    uint32_t pf[4];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const float e0 = fast_exp2(s[t][0] - mu[0]), e1 = fast_exp2(s[t][1] - mu[0]);
      const float e2 = fast_exp2(s[t][2] - mu[1]), e3 = fast_exp2(s[t][3] - mu[1]);
      l[0] += e0 + e1;
      l[1] += e2 + e3;
      // probabilities in bf16 for the tensor core: half a step of 2^-8 each, averaged over the keys
      pf[t * 2] = pack_bf16x2(e0, e1);
      pf[t * 2 + 1] = pack_bf16x2(e2, e3);
    }
#pragma unroll
    for (int t = 0; t < 16; t += 2) {
      uint32_t vf[4];  // keys 0..15 x dims 8 t .. 8 t + 15
      const int row = (lm & 1) * 8 + lr, x = t + (lm >> 1);
      ldsm4_t(vf, vs + (x >> 3) * kBox + row * 128 + (((x & 7) ^ lr) << 4));
      if (part) {  // zero probabilities times what stands in unused rows could be NaN
        vf[0] &= used[0];
        vf[1] &= used[1];
        vf[2] &= used[0];
        vf[3] &= used[1];
      }
      mma16816(o[t], pf, vf[0], vf[1]);
      mma16816(o[t + 1], pf, vf[2], vf[3]);
    }
    __syncwarp();  // every lane is done with the slot
    if (lane == 0 && c + kRing * kWarps < c1) load(c + kRing * kWarps, slot);
    if (++slot == kRing) {
      slot = 0;
      phase ^= 1u;
    }
  }
  if (*abort_flag) {  // a wait ran out: let the copies already issued land before the ring is left
    volatile int never = 0;
    for (int s = 0; s < kRing; ++s)
      if (c0 + s * kWarps < c1) mbar_wait(&full[s], 0, &never, ZI_DEVERR_TIMEOUT_DRAIN, 1000000ull);
    const unsigned long long t0 = globaltimer();
    while (globaltimer() - t0 < 200000ull) {
    }
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
    l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
  }
  __syncthreads();  // the rings become the warps' partials
  float* parts = reinterpret_cast<float*>(smem);
  float* mine = parts + warp * kPartFloats;
#pragma unroll
  for (int t = 0; t < 16; ++t)
#pragma unroll
    for (int h = 0; h < 2; ++h)
      *reinterpret_cast<float2*>(mine + (gid + 8 * h) * 128 + t * 8 + tid * 2) = make_float2(o[t][2 * h], o[t][2 * h + 1]);
  if (tid == 0) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      mine[2048 + gid + 8 * h] = m[h];
      mine[2064 + gid + 8 * h] = l[h];
    }
  }
  __syncthreads();
  // join the warps, warps in order: 8 threads per row, 16 columns each
  float* cta = parts + kWarps * kPartFloats;
  const int live = min(16, rows - row0);
  if (int(threadIdx.x) / 8 < live) {
    const int r = threadIdx.x / 8, x = threadIdx.x % 8;
    float f[kWarps], mm = -INFINITY, ll = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      f[w] = parts[w * kPartFloats + 2048 + r];
      mm = fmaxf(mm, f[w]);
    }
    const float mu = mm == -INFINITY ? 0.f : mm;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      f[w] = fast_exp2(f[w] - mu);
      ll = fmaf(f[w], parts[w * kPartFloats + 2064 + r], ll);
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float4 y = *reinterpret_cast<const float4*>(parts + w * kPartFloats + r * 128 + (c * 8 + x) * 4);
        acc = make_float4(fmaf(f[w], y.x, acc.x), fmaf(f[w], y.y, acc.y), fmaf(f[w], y.z, acc.z), fmaf(f[w], y.w, acc.w));
      }
      *reinterpret_cast<float4*>(cta + r * 128 + (c * 8 + x) * 4) = acc;
    }
    if (x == 0) {
      cta[2048 + r] = mm;
      cta[2064 + r] = ll;
    }
  }
  if (splits > 1) cluster_sync(); else __syncthreads();
  // join the cluster, ranks in order: this CTA's share of the rows' 4-column pieces
  const bool bad = splits > 1 ? any_peer_set(abort_flag, splits) : *abort_flag != 0;
  uint32_t peer[kMaxCluster];
#pragma unroll
  for (int w = 0; w < kMaxCluster; ++w)
    peer[w] = splits > 1 ? peer_addr(smem_u32(cta), w < splits ? w : 0) : smem_u32(cta);
  for (int e = rank + int(threadIdx.x) * splits; e < live * 32 && !bad; e += kThreads * splits) {
    const int r = e >> 5, c = e & 31;
    float f[kMaxCluster], lw[kMaxCluster], mm = -INFINITY, ll = 0.f;
    float4 y[kMaxCluster];
#pragma unroll
    for (int w = 0; w < kMaxCluster; ++w) {
      f[w] = ld_peer(peer[w] + (2048 + r) * 4, w < splits);
      lw[w] = ld_peer(peer[w] + (2064 + r) * 4, w < splits);
      y[w] = ld_peer4(peer[w] + (r * 128 + c * 4) * 4, w < splits);
    }
#pragma unroll
    for (int w = 0; w < kMaxCluster; ++w)
      if (w < splits) mm = fmaxf(mm, f[w]);
    const float mu = mm == -INFINITY ? 0.f : mm;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kMaxCluster; ++w) {
      if (w < splits) {
        f[w] = fast_exp2(f[w] - mu);
        ll = fmaf(f[w], lw[w], ll);
        acc = make_float4(fmaf(f[w], y[w].x, acc.x), fmaf(f[w], y[w].y, acc.y), fmaf(f[w], y[w].z, acc.z),
                          fmaf(f[w], y[w].w, acc.w));
      }
    }
    const int row = row0 + r, i = row / p.group, g = row - i * p.group;
    const float inv = ll > 0.f ? 1.f / ll : 0.f;  // a row that sees no key: 0
    *reinterpret_cast<uint2*>(p.out + b * p.o_bs + i * p.o_rs + (hk * p.group + g) * p.o_hs + c * 4) =
        make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
  }
  if (splits > 1) cluster_sync();  // no CTA leaves while its partial may be read
}

// ------------------------------------------------------------------ many queries
// Flash attention on tcgen05, laid out as attention_kernel is (two 128-row tiles A and B per
// CTA, S and O of both in TMEM, P written back over its S, one softmax thread per row), with
// - a row = one query of one head of a key head's group, packed as for few queries: the
//   heads that share keys share the CTA's K and V tiles, and a causal tile spans fewer queries;
// - Q written to smem by the row threads (any strides), K and V tiles by TMA;
// - key tiles that no row of a row tile sees left out for it (by the rows' limits, and by the
//   ranges of document ids of the key tile and of the rows), elementwise masks only on key
//   tiles that some row sees in part;
// - V rows that no query may see (past the element's keys, or with a negative id) cleared in
//   smem before the product: zero probabilities times NaN would be NaN;
// - with few CTAs, a cluster that shares a unit's keys and joins its partials through
//   distributed shared memory in rank order (no workspace, no atomics).
// Bound by the softmax's latency between a tile's two products: 16,896 tokens x 30 heads with cap and bias 5.76 ms
// (760 TFLOP/s; 3.1 us a step of 256 x 128 scores against 1.1 of MMA); a pack of 4224 in five documents 167 us.
// Warps 0..3 rows of tile A, 4..7 of tile B, 8 K loads, 9 MMA, 10 V loads, 11 clears V.
namespace many {
constexpr int kThreads = 384;
constexpr int kRegsSoftmax = 216, kRegsOther = 56;  // as attention_kernel: 62464 <= 384 x 168 registers at launch
constexpr uint32_t kTile = 128 * 128 * 2, kHalf = kTile / 2;
constexpr int kKSlots = 3, kVSlots = 2;
constexpr uint32_t kQ0 = 0, kK0 = 2 * kTile, kV0 = kK0 + kKSlots * kTile;
constexpr uint32_t kBar = kV0 + kVSlots * kTile;
constexpr int kListTiles = 2048;  // key tiles whose state fits the lists; later ones are masked elementwise
constexpr int kListWords = kListTiles / 32;
constexpr uint32_t kList = kBar + 256;           // bit maps of the key tiles: seen [2 row tiles][kListWords], then full
constexpr uint32_t kSmemBytes = kList + 4 * kListWords * 4 + 1024;
constexpr uint32_t kScan = kK0;                  // ids of each key tile, before the rings are used: lowest, highest, any negative
static_assert(kListTiles * 12 <= kBar - kK0, "the scan fits the rings");
static_assert(kSmemBytes <= 232448, "shared memory");
constexpr uint32_t kColS = 0, kColO = 256;
// the partial of a split unit, over K and V: O [t][32 column quads][128 rows] float4, then (m, l) [256] float2
constexpr uint32_t kPart = kK0;
static_assert(kPart + 2 * 32 * 128 * 16 + 256 * 8 <= kBar, "partials fit the rings");
}  // namespace many

// cap tanh(z) for a pair on the FMA pipe, |z| <= 3/4: z P(z^2) with a degree-7 odd polynomial
// fitted here by the Remez exchange on the absolute error (3.7e-6 at most, and 4.5e-5 of tanh(z)).  c: its
// coefficients times the cap and the powers of the score's factor, so s2 are raw scores.
constexpr float kCapRange = 0.75f;
ZI_DEV uint64_t cap_poly_pair(uint64_t s2, const float* c) {
  const uint64_t u = f2_mul(s2, s2);
  uint64_t r = f2_fma(f2_pack(c[3], c[3]), u, f2_pack(c[2], c[2]));
  r = f2_fma(r, u, f2_pack(c[1], c[1]));
  r = f2_fma(r, u, f2_pack(c[0], c[0]));
  return f2_mul(r, s2);
}

// The low word of a 128-byte-swizzled operand descriptor (smem_desc_sw128); its high word is
// the same for every tile.  Kept opaque to the compiler: it would otherwise hold the sixteen
// descriptors of both Q tiles across the loop, spill them from the MMA warp's 56 registers and
// slow the issue of every MMA (a step of 128 keys without cap: 2.5 us with the spills, 2.2 without).
ZI_DEV uint32_t desc_low(uint32_t saddr, uint32_t lead_bytes) {
  uint32_t lo = ((saddr & 0x3FFFFu) >> 4) | ((lead_bytes >> 4) << 16);
  asm volatile("" : "+r"(lo));
  return lo;
}
ZI_DEV uint64_t desc_at(uint32_t low, uint32_t bytes) {
  constexpr uint32_t kHigh = (1024u >> 4) | (1u << 14) | (2u << 29);
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(low + (bytes >> 4)), "r"(kHigh));
  return d;
}

template <bool CAP, bool BIAS, bool DOC>
__global__ void __launch_bounds__(many::kThreads, 1)
    attention_many_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                          MaskedParams p, int splits) {
  using namespace many;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kBar);
  uint64_t* k_full = bars + 0;    // [kKSlots]
  uint64_t* k_empty = bars + 3;   // [kKSlots]
  uint64_t* v_full = bars + 6;    // [kVSlots]
  uint64_t* v_empty = bars + 8;   // [kVSlots]
  uint64_t* v_clean = bars + 10;  // [kVSlots]
  uint64_t* s_full = bars + 12;   // [2 tiles]
  uint64_t* p_full = bars + 14;   // [2 tiles]
  uint64_t* pv_done = bars + 16;  // [2 tiles]
  uint64_t* drain = bars + 18;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 19);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* lim_min = reinterpret_cast<int*>(tmem_slot + 2);  // of the rows of tile A, of tile B (all arrays below likewise)
  int* lim_max = lim_min + 2;
  int* doc_min = lim_min + 4;  // of the rows' ids that are not negative ...
  int* doc_max = lim_min + 6;
  int* doc_neg = lim_min + 8;  // ... and whether any is
  uint32_t* seen = reinterpret_cast<uint32_t*>(smem + kList);  // [2][kListWords] some row of the row tile sees some key ...
  uint32_t* full = seen + 2 * kListWords;                      // ... every row every key

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // Blocks: rank fastest, then the key heads (of all batch elements) of a group, then the 256-row units from the
  // end: the longest ones (a causal mask's last rows, a pack's texts behind its images, which see several
  // documents) start first.  Groups are as many heads as keep their K and V in L2 (p.head_group).
  const int rank = int(blockIdx.x) % splits;
  const int rows = p.q_len * p.group;
  const int units = (rows + 255) / 256;
  const int in_group = int(blockIdx.x) / splits % (units * p.head_group);
  const int hb0 = int(blockIdx.x) / splits / (units * p.head_group) * p.head_group;
  const int hb_n = min(p.head_group, p.kv_heads * p.batch - hb0);
  const int hb = hb0 + in_group % hb_n;
  const int hk = hb % p.kv_heads, b = hb / p.kv_heads;
  const int row0 = (units - 1 - in_group / hb_n) * 256;
  const int n = masked_keys(p, b);

  if (threadIdx.x == 0) {
    for (int i = 0; i < kKSlots; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&k_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&v_full[i], 1);
      mbar_init(&v_empty[i], 1);
      mbar_init(&v_clean[i], 1);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);  // one arrival per softmax warp
      mbar_init(&pv_done[i], 1);
    }
    mbar_init(drain, 1);
    *abort_flag = device_error_set() ? 1 : 0;  // an earlier kernel timed out: leave everything untouched
    for (int t = 0; t < 2; ++t) {
      lim_min[t] = 0x7fffffff;
      lim_max[t] = 0;
      doc_min[t] = 0x7fffffff;
      doc_max[t] = -1;
      doc_neg[t] = 0;
    }
    fence_mbar_init();
  }
  if (warp == 8 && lane == 0) {
    prefetch_tmap(&tmK);
    prefetch_tmap(&tmV);
  }
  if (warp == 9) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const bool skip = *abort_flag != 0;

  const int* kd = DOC ? p.k_doc + size_t(b) * p.kv_len : nullptr;
  int* scan = reinterpret_cast<int*>(smem + kScan);
  // Ranges of the document ids of key tiles first, first + step, ... below end; three tiles' loads on their way per warp
  auto scan_ids = [&](int first, int step, int end) {
    constexpr int kAhead = 3;
    for (int j = first; j < end; j += step * kAhead) {
      int d[kAhead][4];
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int key = (j + u * step) * 128 + e * 32 + lane;
          d[u][e] = key < n ? __ldg(kd + key) : -1;
        }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        int lo = 0x7fffffff, hi = -1, neg = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (d[u][e] < 0) neg = 1;
          else lo = min(lo, d[u][e]);
          hi = max(hi, d[u][e]);
        }
        lo = __reduce_min_sync(0xffffffffu, lo);
        hi = __reduce_max_sync(0xffffffffu, hi);
        neg = __reduce_max_sync(0xffffffffu, neg);
        const int jj = j + u * step;
        if (lane == 0 && jj < end) {
          scan[jj] = lo;
          scan[kListTiles + jj] = hi;
          scan[2 * kListTiles + jj] = neg;
        }
      }
    }
  };
  // key tiles to scan: those that the CTA's last row may see (limits grow with the row).  The first ones by the
  // warps that load no Q, meanwhile.
  const int scan_n = DOC ? min(kListTiles, (masked_limit(p, b, (min(row0 + 256, rows) - 1) / p.group, n) + 127) / 128) : 0;
  const int scan_early = min(scan_n, 36);
  if (DOC && warp >= 8) scan_ids(warp - 8, 4, scan_early);

  // the row threads: their warp's 32 rows of Q to smem (half a warp per row, 256 contiguous bytes, all loads on
  // their way at once), and what their own row sees
  const int row = row0 + int(threadIdx.x);
  const int qi = row / p.group, qg = row - qi * p.group;
  int lim = 0, doc = 0;
  if (warp < 8) {
    const bool have = row < rows;
    const long long at = have ? b * p.q_bs + qi * p.q_rs + (hk * p.group + qg) * p.q_hs : -1;
    const int x = lane & 15;
    uint4 w[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const long long src = __shfl_sync(0xffffffffu, at, 2 * e + (lane >> 4));
      w[e] = __ldg(reinterpret_cast<const uint4*>(p.q + (src < 0 ? 0 : src)) + x);
    }
    int d_lo = 0x7fffffff, d_hi = -1, neg = 0;
    if (have) {
      lim = masked_limit(p, b, qi, n);
      if (DOC) {
        doc = __ldg(p.q_doc + size_t(b) * p.q_len + qi);
        if (doc < 0) {
          lim = 0;
          neg = 1;
        } else {
          d_lo = d_hi = doc;
        }
      }
    }
    const int lo = __reduce_min_sync(0xffffffffu, have ? lim : 0x7fffffff);
    const int hi = __reduce_max_sync(0xffffffffu, lim);
    d_lo = __reduce_min_sync(0xffffffffu, d_lo);
    d_hi = __reduce_max_sync(0xffffffffu, d_hi);
    neg = __reduce_max_sync(0xffffffffu, neg);
    if (lane == 0) {
      const int t = warp >> 2;
      atomicMin(lim_min + t, lo);
      atomicMax(lim_max + t, hi);
      atomicMin(doc_min + t, d_lo);
      atomicMax(doc_max + t, d_hi);
      atomicMax(doc_neg + t, neg);
    }
    const int live = rows - (row0 + warp * 32);  // rows past the end are zeros
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const int r = 2 * e + (lane >> 4), i = (warp & 3) * 32 + r;
      *reinterpret_cast<uint4*>(smem + kQ0 + (warp >> 2) * kTile + (x >> 3) * kHalf + i * 128 +
                                (((x & 7) ^ (i & 7)) << 4)) = r < live ? w[e] : make_uint4(0, 0, 0, 0);
    }
    fence_proxy_async_smem();
  }
  __syncthreads();
  const int tiles_a = (lim_max[0] + 127) / 128, tiles_b = (lim_max[1] + 127) / 128;  // key tiles that any of their rows may see
  const int full_a = lim_min[0] / 128, full_b = lim_min[1] / 128;                    // ... that all see, by their limits
  const int tiles = max(tiles_a, tiles_b);
  const int my_j0 = int(static_cast<long long>(rank) * tiles / splits);
  const int my_j1 = int(static_cast<long long>(rank + 1) * tiles / splits);
  if constexpr (DOC) {
    if (scan_early < scan_n) {
      scan_ids(scan_early + warp, kThreads / 32, scan_n);
      __syncthreads();
    }
    for (int j0 = warp * 32; j0 < scan_n; j0 += kThreads) {
      const int j = j0 + lane, jj = min(j, scan_n - 1);
      const int lo = scan[jj], hi = scan[kListTiles + jj], neg = scan[2 * kListTiles + jj];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const bool some = j < (t ? tiles_b : tiles_a) && hi >= doc_min[t] && lo <= doc_max[t];
        const bool every = !neg && !doc_neg[t] && lo == hi && lo == doc_min[t] && lo == doc_max[t] && j < (t ? full_b : full_a);
        const uint32_t ws = __ballot_sync(0xffffffffu, some), wf = __ballot_sync(0xffffffffu, every);
        if (lane == 0) {
          seen[t * kListWords + j0 / 32] = ws;
          full[t * kListWords + j0 / 32] = wf;
        }
      }
    }
    fence_proxy_async_smem();  // the scan's place goes to the TMA loads
    __syncthreads();
  }
  // what row tile t sees of key tile j: 0 nothing, 1 every row every key, 2 between
  auto state = [&](int t, int j) -> uint32_t {
    if (j >= (t ? tiles_b : tiles_a)) return 0u;
    if (!DOC) return j < (t ? full_b : full_a) ? 1u : 2u;
    if (j >= kListTiles) return 2u;
    const int w = t * kListWords + (j >> 5);
    return seen[w] >> (j & 31) & 1u ? (full[w] >> (j & 31) & 1u ? 1u : 2u) : 0u;
  };
  // the next key tile of this CTA at or after j that some row of the row tiles in `which` (bit 0 A, bit 1 B) sees;
  // at or past my_j1: none
  auto next = [&](int j, int which) -> int {
    if constexpr (DOC) {
      while (j < my_j1 && j < kListTiles) {
        const uint32_t w = ((which & 1 ? seen[j >> 5] : 0u) | (which & 2 ? seen[kListWords + (j >> 5)] : 0u)) >> (j & 31);
        if (w) return j + __ffs(w) - 1;
        j = (j | 31) + 1;
      }
    }
    return j;
  };
  const int first = skip ? my_j1 : next(my_j0, 3);
  const bool clean = DOC || p.lengths != nullptr;  // V may hold rows that nobody sees

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
    if (warp == 8 || warp == 10) {
      if (lane == 0) {
        const bool kq = warp == 8;
        uint64_t* fullb = kq ? k_full : v_full;
        uint64_t* emptyb = kq ? k_empty : v_empty;
        const CUtensorMap* map = kq ? &tmK : &tmV;
        const uint32_t base = kq ? kK0 : kV0;
        const int nslots = kq ? kKSlots : kVSlots;
        int it = 0;
        bool ok = true;
        for (int j = first; j < my_j1; j = next(j + 1, 3), ++it) {
          const int bi = it % nslots;
          if (!mbar_wait(&emptyb[bi], (uint32_t(it / nslots) & 1u) ^ 1u, abort_flag, ZI_DEVERR_TIMEOUT_PRODUCER)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&fullb[bi], kTile);
          tma_load_4d(smem + base + bi * kTile, map, &fullb[bi], 0, hk, j * 128, b);
          tma_load_4d(smem + base + bi * kTile + kHalf, map, &fullb[bi], 64, hk, j * 128, b);
        }
        if (!ok) {
          volatile int never = 0;
          for (int k = it > nslots ? it - nslots : 0; k < it; ++k)
            mbar_wait(&fullb[k % nslots], uint32_t(k / nslots) & 1u, &never, ZI_DEVERR_TIMEOUT_DRAIN);
        }
      }
    } else if (warp == 9) {
      if (lane == 0 && first < my_j1) {
        constexpr uint32_t idesc_s = idesc_bf16_f32(128, 128, false, false);
        constexpr uint32_t idesc_o = idesc_bf16_f32(128, 128, false, true);
        auto issue_s = [&](int t, int it) {
          const uint32_t q_low = desc_low(smem_u32(smem + kQ0 + t * kTile), 16);
          const uint32_t k_low = desc_low(smem_u32(smem + kK0 + (it % kKSlots) * kTile), 16);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const uint32_t at = (k >> 2) * kHalf + (k & 3) * 32;
            tc_mma(tmem + kColS + 128 * t, desc_at(q_low, at), desc_at(k_low, at), idesc_s, k > 0 ? 1u : 0u);
          }
          tc_commit(&s_full[t]);
        };
        // done: products of tile t so far
        auto issue_pv = [&](int t, int it, int done) -> bool {
          if (!mbar_wait(&p_full[t], uint32_t(done) & 1u, abort_flag, ZI_DEVERR_TIMEOUT_MMA)) return false;
          tc_fence_after();
          const uint32_t v_low = desc_low(smem_u32(smem + kV0 + (it & 1) * kTile), kHalf);
#pragma unroll
          for (int k = 0; k < 8; ++k)
            tc_mma_ts(tmem + kColO + 128 * t, tmem + kColS + 128 * t + 8 * k, desc_at(v_low, k * 2048), idesc_o,
                      (done > 0 || k > 0) ? 1u : 0u);
          tc_commit(&pv_done[t]);
          return true;
        };
        auto wait_k = [&](int it) {
          return mbar_wait(&k_full[it % kKSlots], uint32_t(it / kKSlots) & 1u, abort_flag, ZI_DEVERR_TIMEOUT_MMA);
        };
        auto wait_v = [&](int it) {
          const uint32_t phase = (uint32_t(it) >> 1) & 1u;
          return mbar_wait(&v_full[it & 1], phase, abort_flag, ZI_DEVERR_TIMEOUT_MMA) &&
                 (!clean || mbar_wait(&v_clean[it & 1], phase, abort_flag, ZI_DEVERR_TIMEOUT_MMA));
        };
        // S_A(0), S_B(0), then O_A += P_A(i) V, S_A(i + 1), O_B += P_B(i) V, S_B(i + 1), each tile where it sees the keys
        bool need_a = state(0, first) != 0, need_b = state(1, first) != 0;
        bool ok = wait_k(0);
        if (ok) {
          tc_fence_after();
          if (need_a) issue_s(0, 0);
          if (need_b) issue_s(1, 0);
          tc_commit(&k_empty[0]);
        }
        int it = 0, done_a = 0, done_b = 0;
        for (int j = first; j < my_j1 && ok; ++it) {
          const int nx = next(j + 1, 3);
          const bool more = nx < my_j1;
          const bool then_a = more && state(0, nx) != 0, then_b = more && state(1, nx) != 0;
          if (!wait_v(it)) { ok = false; break; }
          if (need_a && !issue_pv(0, it, done_a++)) { ok = false; break; }
          if (more) {
            if (!wait_k(it + 1)) { ok = false; break; }
            tc_fence_after();
            if (then_a) issue_s(0, it + 1);
          }
          if (need_b && !issue_pv(1, it, done_b++)) { ok = false; break; }
          tc_commit(&v_empty[it & 1]);
          if (more) {
            if (then_b) issue_s(1, it + 1);
            tc_commit(&k_empty[(it + 1) % kKSlots]);
          }
          need_a = then_a;
          need_b = then_b;
          j = nx;
        }
        if (!ok) {
          tc_commit(drain);
          volatile int never = 0;
          mbar_wait(drain, 0, &never, ZI_DEVERR_TIMEOUT_DRAIN);
        }
      }
    } else if (clean) {
      int it = 0;
      for (int j = first; j < my_j1; j = next(j + 1, 3), ++it) {
        uint32_t dirty = 0;  // bit e: nobody sees key j 128 + e 32 + lane
        if (state(0, j) != 1 || state(1, j) != 1) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int key = j * 128 + e * 32 + lane;
            dirty |= (key >= n || (DOC && __ldg(kd + key) < 0) ? 1u : 0u) << e;
          }
        }
        if (!mbar_wait_warp(&v_full[it & 1], (uint32_t(it) >> 1) & 1u, abort_flag, ZI_DEVERR_TIMEOUT_SOFTMAX)) break;
        if (__any_sync(0xffffffffu, dirty != 0)) {
          uint8_t* v = smem + kV0 + (it & 1) * kTile;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int r = e * 32 + lane;
            if (dirty >> e & 1u) {
#pragma unroll
              for (int x = 0; x < 8; ++x) {
                *reinterpret_cast<uint4*>(v + r * 128 + x * 16) = make_uint4(0, 0, 0, 0);
                *reinterpret_cast<uint4*>(v + kHalf + r * 128 + x * 16) = make_uint4(0, 0, 0, 0);
              }
            }
          }
          fence_proxy_async_smem();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&v_clean[it & 1]);
      }
    }
    __syncwarp();
    if (splits > 1) {
      cluster_sync();
      cluster_sync();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    const int t = warp >> 2, q = warp & 3;
    const int i = q * 32 + lane;
    const uint32_t lane_addr = tmem + (uint32_t(q * 32) << 16);
    const uint32_t s_addr = lane_addr + kColS + 128 * t;
    const uint32_t o_addr = lane_addr + kColO + 128 * t;
    float m_run = -INFINITY, l = 0.f;
    bool ok = !skip;
    // A wait of this lane ran out: it goes on with what TMEM holds until the next vote, where its warp leaves together
    // (a vote at each wait costs 3% of the kernel)
    bool lost = false;
    int it = 0;
    {
      // scores are in the exp2 domain after a cap, and scaled into it by the exponential's argument without one
      const float sl2 = CAP ? 1.f : p.scale_log2;
      float slope = 0.f, pos = 0.f;
      int pos_lo = 0, pos_hi = 0;  // places of the warp's first and last row
      if constexpr (BIAS) {
        const int r = min(row, rows - 1), ri = r / p.group;
        slope = __ldg(p.slopes + hk * p.group + r - ri * p.group) * (1.4426950408889634f / sl2);
        pos = float(ri + n - p.q_len);
        pos_lo = __shfl_sync(0xffffffffu, ri, 0) + n - p.q_len;
        pos_hi = __shfl_sync(0xffffffffu, ri, 31) + n - p.q_len;
      }
      float cc[4];
      if constexpr (CAP) {
        const float z1 = p.scale_log2, z2 = z1 * z1, y1 = z1 * p.cap_log2;
        cc[0] = 0.9999556008f * y1;
        cc[1] = -0.3322276376f * y1 * z2;
        cc[2] = 0.1257709249f * y1 * z2 * z2;
        cc[3] = -0.0337782849f * y1 * z2 * z2 * z2;
      }
      uint32_t s[128];
      const int mine = 1 << t, stop = min(my_j1, t ? tiles_b : tiles_a);
      for (int j = next(my_j0, mine); ok && j < stop; j = next(j + 1, mine)) {
        const bool part = state(t, j) != 1;
        int id[4];  // document ids of keys w 32 + lane, on their way while S is computed
        if (DOC && part) {
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const int key = j * 128 + w * 32 + lane;
            id[w] = key < n ? __ldg(kd + key) : -1;
          }
        }
        lost |= !mbar_wait(&s_full[t], uint32_t(it) & 1u, abort_flag, ZI_DEVERR_TIMEOUT_SOFTMAX);
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(s_addr + c * 32, &s[c * 32]);
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < 4; ++c) reg_fence32(&s[c * 32]);
        // bit c of vis: the row sees key j 128 + c
        uint32_t vis[4];
        auto see = [&]() {
          const int left = lim - j * 128;
#pragma unroll
          for (int w = 0; w < 4; ++w) vis[w] = left >= 32 * w + 32 ? ~0u : left <= 32 * w ? 0u : (1u << (left - 32 * w)) - 1u;
        };
        if constexpr (DOC) {
          if (part) {
            see();
            for (uint32_t todo = ~0u; todo;) {  // once for each document among the warp's rows
              const int d = __shfl_sync(0xffffffffu, doc, __ffs(todo) - 1);
              todo &= ~__ballot_sync(0xffffffffu, doc == d);
#pragma unroll
              for (int w = 0; w < 4; ++w) {
                const uint32_t same = __ballot_sync(0xffffffffu, id[w] == d);
                if (doc == d) vis[w] &= same;
              }
            }
          }
        }
        if constexpr (CAP) {
          // |z| within the polynomial's range over the keys that the row sees, or (scores near the cap and past it)
          // through exp and a reciprocal; each row by its own keys alone, whatever its neighbours and hidden keys hold.
          // A NaN, of a key row that nobody sees, stays in its column and is masked below.
          float mx4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int c = 0; c < 128; c += 2)
            mx4[c / 2 & 3] = max3f(mx4[c / 2 & 3], fabsf(__uint_as_float(s[c])), fabsf(__uint_as_float(s[c + 1])));
          float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));
          bool near = p.cap_poly && mx * p.scale_log2 <= kCapRange;
          auto poly = [&]() {
#pragma unroll
            for (int c = 0; c < 64; ++c) {
              float y0, y1;
              f2_unpack(cap_poly_pair(f2_pack(__uint_as_float(s[2 * c]), __uint_as_float(s[2 * c + 1])), cc), y0, y1);
              s[2 * c] = __float_as_uint(y0);
              s[2 * c + 1] = __float_as_uint(y1);
            }
          };
          if (__builtin_expect(__all_sync(0xffffffffu, near), 1)) {
            poly();
          } else {
            if (part && p.cap_poly && !near) {  // perhaps by hidden keys alone
              if constexpr (!DOC) see();
              mx = 0.f;
#pragma unroll
              for (int c = 0; c < 128; ++c)
                if (vis[c >> 5] >> (c & 31) & 1u) mx = fmaxf(mx, fabsf(__uint_as_float(s[c])));
              near = mx * p.scale_log2 <= kCapRange;
            }
            if (near) {
              poly();
            } else {
#pragma unroll
              for (int c = 0; c < 128; ++c)
                s[c] = __float_as_uint(tanh_score(__uint_as_float(s[c]) * p.scale_log2) * p.cap_log2);
            }
            __syncwarp();
          }
        }
        float base = 0.f;  // what every score of the row in this tile still lacks, in the exp2 domain
        if constexpr (BIAS) {
          const float away = pos - float(j * 128);
          const bool below = j * 128 + 127 <= pos_lo;
          if (below || j * 128 >= pos_hi) {
            // every key on one side of every row of the warp: |p_i - j| is linear, its row part goes to the base
            const float sg = below ? slope : -slope;
            base = -sg * away * sl2;
#pragma unroll
            for (int c = 0; c < 128; ++c) s[c] = __float_as_uint(fmaf(sg, float(c), __uint_as_float(s[c])));
          } else {
#pragma unroll
            for (int c = 0; c < 128; ++c)
              s[c] = __float_as_uint(fmaf(-slope, fabsf(away - float(c)), __uint_as_float(s[c])));
          }
        }
        if (part) {
          if constexpr (!DOC) see();
#pragma unroll
          for (int c = 0; c < 128; ++c)
            if (!(vis[c >> 5] >> (c & 31) & 1u)) s[c] = __float_as_uint(-INFINITY);
        }
        float mx8[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) mx8[k] = __uint_as_float(s[k]);
#pragma unroll
        for (int c = 8; c < 120; c += 16) {
#pragma unroll
          for (int k = 0; k < 8; ++k) mx8[k] = max3f(mx8[k], __uint_as_float(s[c + k]), __uint_as_float(s[c + 8 + k]));
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) mx8[k] = fmaxf(mx8[k], __uint_as_float(s[120 + k]));
        const float mx = max3f(max3f(mx8[0], mx8[1], mx8[2]), max3f(mx8[3], mx8[4], mx8[5]), fmaxf(mx8[6], mx8[7]));
        const float m_new = fmaxf(m_run, fmaf(mx, sl2, base));
        // each row moves its maximum by its own scores alone, so its result does not depend on its neighbours
        const bool grows = m_new > m_run + 8.0f;
        const bool resc = __any_sync(0xffffffffu, grows || lost);
        if (resc && __any_sync(0xffffffffu, lost)) {
          ok = false;
          break;
        }
        float alpha = 1.0f;
        if (grows) {
          alpha = m_run == -INFINITY ? 0.f : fast_exp2(m_run - m_new);  // a row that has seen nothing yet holds nothing
          m_run = m_new;
          l *= alpha;
        }
        const float m_use = m_run == -INFINITY ? 0.f : m_run;
        const uint64_t sl2x2 = f2_pack(sl2, sl2), negm = f2_pack(base - m_use, base - m_use);
        uint64_t sum2[4] = {0, 0, 0, 0};
        uint32_t pw[64];
#pragma unroll
        for (int c = 0; c < 64; ++c) {
          float x0, x1;
          const uint64_t s2 = f2_pack(__uint_as_float(s[2 * c]), __uint_as_float(s[2 * c + 1]));
          f2_unpack(CAP ? f2_add(s2, negm) : f2_fma(s2, sl2x2, negm), x0, x1);
          float e0, e1;
          if (!CAP && ((c & 7) == 1 || (c & 7) == 4 || (c & 7) == 6)) {  // 3 of 8 pairs on the FMA pipe; the cap fills it
            exp2_poly_pair(x0, x1, e0, e1);
          } else {
            e0 = fast_exp2(x0);
            e1 = fast_exp2(x1);
          }
          sum2[c & 3] = f2_add(sum2[c & 3], f2_pack(e0, e1));
          pw[c] = pack_bf16x2(e0, e1);
        }
        {
          float a0, a1, b0, b1, c0, c1, d0, d1;
          f2_unpack(sum2[0], a0, a1);
          f2_unpack(sum2[1], b0, b1);
          f2_unpack(sum2[2], c0, c1);
          f2_unpack(sum2[3], d0, d1);
          l += ((a0 + a1) + (b0 + b1)) + ((c0 + c1) + (d0 + d1));
        }
        if (resc && it > 0) {
          lost |= !mbar_wait(&pv_done[t], uint32_t(it - 1) & 1u, abort_flag, ZI_DEVERR_TIMEOUT_SOFTMAX);
          tc_fence_after();
          const uint64_t a2 = f2_pack(alpha, alpha);
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t o[32];
            tmem_ld32_sync(o_addr + c * 32, o);
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              float y0, y1;
              f2_unpack(f2_mul(f2_pack(__uint_as_float(o[2 * k]), __uint_as_float(o[2 * k + 1])), a2), y0, y1);
              o[2 * k] = __float_as_uint(y0);
              o[2 * k + 1] = __float_as_uint(y1);
            }
            tmem_st32(o_addr + c * 32, o);
          }
        }
        tmem_st32(s_addr, &pw[0]);
        tmem_st32(s_addr + 32, &pw[32]);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[t]);  // for the whole warp: its stores are complete
        ++it;
      }
      if (ok && it > 0) {
        ok = !__any_sync(0xffffffffu, lost) && mbar_wait_warp(&pv_done[t], uint32_t(it - 1) & 1u, abort_flag, ZI_DEVERR_TIMEOUT_SOFTMAX);
        if (ok) tc_fence_after();
      }
    }
    const bool live = row < rows;
    uint16_t* orow = p.out + b * p.o_bs + qi * p.o_rs + (hk * p.group + qg) * p.o_hs;
    if (splits == 1) {
      const float inv = m_run == -INFINITY ? 0.f : 1.0f / l;  // a row that sees no key: zeros
      if (ok) {
        // Through this warp's quarter of its tile's Q (read for the last time by an MMA that is done), so that half a
        // warp stores a row's 256 bytes: a thread storing its own row touches 32 lines with every instruction
        uint8_t* stage = smem + kQ0 + t * kTile + q * 8192;
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          uint32_t o[32];
          if (it > 0) tmem_ld32_sync(o_addr + c * 32, o);
          float f[32];
#pragma unroll
          for (int k = 0; k < 32; ++k) f[k] = it > 0 ? __uint_as_float(o[k]) * inv : 0.f;
#pragma unroll
          for (int k = 0; k < 4; ++k)
            *reinterpret_cast<uint4*>(stage + lane * 256 + (((c * 4 + k) ^ (lane & 7)) << 4)) =
                make_uint4(pack_bf16x2(f[8 * k], f[8 * k + 1]), pack_bf16x2(f[8 * k + 2], f[8 * k + 3]),
                           pack_bf16x2(f[8 * k + 4], f[8 * k + 5]), pack_bf16x2(f[8 * k + 6], f[8 * k + 7]));
        }
        __syncwarp();
        const long long at = orow - p.out;
        const int x = lane & 15, left = rows - (row - lane);  // rows of the warp that exist
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int r = 2 * e + (lane >> 4);
          const long long to = __shfl_sync(0xffffffffu, at, r);
          const uint4 w = *reinterpret_cast<const uint4*>(stage + r * 256 + ((x ^ (r & 7)) << 4));
          if (r < left) *reinterpret_cast<uint4*>(p.out + to + x * 8) = w;
        }
      }
    } else {
      // leave the partial in this CTA's smem, once both tiles' last products are done: the rings are free then, every
      // load was consumed by one ...
      asm volatile("bar.sync 1, 256;" ::: "memory");
      float4* part = reinterpret_cast<float4*>(smem + kPart);
      float2* ml = reinterpret_cast<float2*>(smem + kPart + 2 * 32 * 128 * 16);
      if (ok) {
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          uint32_t o[32];
          if (it > 0) tmem_ld32_sync(o_addr + c * 32, o);
#pragma unroll
          for (int k = 0; k < 8; ++k)
            part[(t * 32 + c * 8 + k) * 128 + i] =
                it > 0 ? make_float4(__uint_as_float(o[4 * k]), __uint_as_float(o[4 * k + 1]),
                                     __uint_as_float(o[4 * k + 2]), __uint_as_float(o[4 * k + 3]))
                       : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        ml[t * 128 + i] = make_float2(m_run, l);
      }
      __syncwarp();
      cluster_sync();
      // ... and join this rank's share of the columns of every row, ranks in order
      if (!any_peer_set(abort_flag, splits) && live) {
        uint32_t peer[kMaxCluster];
        float w[kMaxCluster], lw[kMaxCluster], mm = -INFINITY, ll = 0.f;
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r) {
          peer[r] = peer_addr(smem_u32(smem + kPart), r < splits ? r : 0);
          const uint32_t at = peer[r] + 2 * 32 * 128 * 16 + (t * 128 + i) * 8;
          w[r] = ld_peer(at, r < splits);
          lw[r] = ld_peer(at + 4, r < splits);
        }
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r)
          if (r < splits) mm = fmaxf(mm, w[r]);
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r) {
          w[r] = r >= splits || w[r] == -INFINITY ? 0.f : fast_exp2(w[r] - mm);
          ll = fmaf(w[r], lw[r], ll);
        }
        const float inv = mm == -INFINITY ? 0.f : 1.0f / ll;
        for (int c = rank * 32 / splits; c < (rank + 1) * 32 / splits; ++c) {
          float4 x[kMaxCluster];
#pragma unroll
          for (int r = 0; r < kMaxCluster; ++r) x[r] = ld_peer4(peer[r] + ((t * 32 + c) * 128 + i) * 16, r < splits);
          float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int r = 0; r < kMaxCluster; ++r)
            a = make_float4(fmaf(w[r], x[r].x, a.x), fmaf(w[r], x[r].y, a.y), fmaf(w[r], x[r].z, a.z), fmaf(w[r], x[r].w, a.w));
          *reinterpret_cast<uint2*>(orow + 4 * c) =
              make_uint2(pack_bf16x2(a.x * inv, a.y * inv), pack_bf16x2(a.z * inv, a.w * inv));
        }
      }
      __syncwarp();
      cluster_sync();  // no CTA leaves while its partial may be read
    }
  }

  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace zi
