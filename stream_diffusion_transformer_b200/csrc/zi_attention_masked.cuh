// Attention with capped scores, a distance bias and masks (head_dim 128, bf16 in and out,
// fp32 scores and softmax):
//   s_ij = scale q_i . k_j;  s = cap tanh(s / cap) (cap > 0);  s -= slope_h |p_i - j|;
//   o_i = sum_j softmax_j(s_ij) v_j over the keys j that query i sees, 0 if it sees none,
// where element b has n_b keys, its queries are the last of them (p_i = i + n_b - q_len),
// and i sees j when j < n_b, and (causal) j <= p_i or j < prefix_b, and (documents) their
// ids are equal and not negative.
#pragma once
#include "zi_common.cuh"

namespace zi {

struct MaskedParams {
  const uint16_t *q, *k, *v;
  uint16_t* out;
  long long q_bs, q_rs, q_hs, k_bs, k_rs, k_hs, v_bs, v_rs, v_hs, o_bs, o_rs, o_hs;  // strides in elements
  int batch, heads, kv_heads, group, q_len, kv_len;
  float scale_log2;     // scale * log2(e); with a cap: scale / cap
  float cap_log2;       // cap * log2(e), 0 = no cap
  const float* slopes;  // [heads] or null
  int causal;
  const int* prefix;    // [batch] or null
  const int* lengths;   // [batch] or null
  const int *q_doc, *k_doc;  // [batch, q_len], [batch, kv_len], or null
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

// tanh(x) = 1 - 2 / (e^2x + 1): an absolute error of a few 2^-24, which a cap of 50 turns
// into 10^-5 of a score.  Infinite e^2x gives 1, e^2x = 0 gives -1.
ZI_DEV float tanh_exp(float x) {
  return 1.f - 2.f * fast_rcp(fast_exp2(x * 2.885390081777927f) + 1.f);
}

// ------------------------------------------------------------------ few queries
// One CTA per 16 rows of a key head (a row is one query of one head of the group, row =
// query * group + head in the group) and share of the keys; a cluster of CTAs shares a
// tile's keys.  Bound by reading K and V: each of the 4 warps streams its own chunks of 32
// keys through a private smem ring with cp.async (3 chunks of K and V deep, 48 KB per
// warp), takes scores and products with mma.sync m16n8k16 (16 rows padded: the tensor work
// is small beside the loads) and keeps its own running maximum and sum.  The warps' and
// then the cluster's partials are joined in a fixed order.
namespace few {
constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kChunk = 32;                       // keys per chunk
constexpr int kRing = 3;
constexpr uint32_t kHalfBytes = kChunk * 256;    // K or V of a chunk: 32 rows of 256 bytes
constexpr uint32_t kChunkBytes = 2 * kHalfBytes;
constexpr uint32_t kWarpBytes = kRing * kChunkBytes;
constexpr uint32_t kSmemBytes = kWarps * kWarpBytes;
constexpr uint32_t kPartFloats = 16 * 128 + 32;  // O [16][128], then m [16], l [16]
static_assert(kWarps * kPartFloats * 4 + kPartFloats * 4 <= kSmemBytes, "partials reuse the ring");
}  // namespace few

ZI_DEV void cp_async16(uint32_t dst, const void* src, bool have) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(have ? 16 : 0) : "memory");
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

__global__ void __launch_bounds__(few::kThreads) attention_few_kernel(MaskedParams p, int splits) {
  using namespace few;
  extern __shared__ __align__(128) uint8_t ring[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = int(blockIdx.x) % splits, tile = int(blockIdx.x) / splits;
  const int hk = blockIdx.y, b = blockIdx.z;
  const int rows = p.q_len * p.group;
  const int row0 = tile * 16;
  const int n = masked_keys(p, b);
  // keys that any row of the tile may see: limits grow with the query
  const int i_last = (min(row0 + 16, rows) - 1) / p.group;
  const int end = masked_limit(p, b, i_last, n);
  const int chunks = (end + kChunk - 1) / kChunk;
  const int c0 = int(static_cast<long long>(rank) * chunks / splits);
  const int c1 = int(static_cast<long long>(rank + 1) * chunks / splits);

  // this lane's two rows (fragment rows lane / 4 and lane / 4 + 8)
  int lim[2], pos[2], doc[2];
  float slope[2];
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
  }
  // Q fragments: 8 steps of 16 dims
  uint32_t qf[8][4];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int r = row0 + gid + 8 * h;
    const int i = r / p.group, g = r - i * p.group;
    const uint16_t* src = p.q + b * p.q_bs + i * p.q_rs + (hk * p.group + g) * p.q_hs;
#pragma unroll
    for (int s = 0; s < 8; ++s) {
      qf[s][h] = r < rows ? *reinterpret_cast<const uint32_t*>(src + s * 16 + tid * 2) : 0u;
      qf[s][2 + h] = r < rows ? *reinterpret_cast<const uint32_t*>(src + s * 16 + 8 + tid * 2) : 0u;
    }
  }
  const uint16_t* kb = p.k + b * p.k_bs + hk * p.k_hs;
  const uint16_t* vb = p.v + b * p.v_bs + hk * p.v_hs;
  const int* kd = p.k_doc ? p.k_doc + size_t(b) * p.kv_len : nullptr;
  const uint32_t base = smem_u32(ring) + warp * kWarpBytes;

  // Chunk c of this warp: rows of 16 16-byte pieces, piece x of row r at slot x ^ (r & 7).  Keys past the
  // element's end are filled with zeros, so whatever stands there never meets a product.
  auto load = [&](int c, int slot) {
    const int key0 = c * kChunk;
    const int half = lane >> 4, x = lane & 15;
#pragma unroll
    for (int r = 0; r < kChunk; r += 2) {
      const int row = r + half, key = key0 + row;
      const bool have = key < n && (!kd || __ldg(kd + key) >= 0);
      const size_t kk = have ? key : 0;
      const uint32_t dst = base + slot * kChunkBytes + row * 256 + ((x ^ (row & 7)) << 4);
      cp_async16(dst, kb + kk * p.k_rs + x * 8, have);
      cp_async16(dst + kHalfBytes, vb + kk * p.v_rs + x * 8, have);
    }
  };

  float o[16][4];
#pragma unroll
  for (int t = 0; t < 16; ++t) o[t][0] = o[t][1] = o[t][2] = o[t][3] = 0.f;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

  int c = c0 + warp;
#pragma unroll
  for (int s = 0; s < kRing - 1; ++s) {
    if (c + s * kWarps < c1) load(c + s * kWarps, s);
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  for (int slot = 0; c < c1; c += kWarps) {
    const int ahead = c + (kRing - 1) * kWarps;
    if (ahead < c1) load(ahead, slot == 0 ? kRing - 1 : slot - 1);
    asm volatile("cp.async.commit_group;" ::: "memory");
    asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 1) : "memory");
    __syncwarp();
    const uint32_t ks = base + slot * kChunkBytes, vs = ks + kHalfBytes;
    slot = slot + 1 == kRing ? 0 : slot + 1;
    float s[4][4];
#pragma unroll
    for (int t = 0; t < 4; ++t) s[t][0] = s[t][1] = s[t][2] = s[t][3] = 0.f;
    const int lr = lane & 7, lm = lane >> 3;  // ldmatrix: this lane's row in matrix lm
#pragma unroll
    for (int kp = 0; kp < 4; ++kp) {  // two 16-dim steps at a time
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        uint32_t kf[4];
        ldsm4(kf, ks + (t * 8 + lr) * 256 + (((kp * 4 + lm) ^ lr) << 4));
        mma16816(s[t], qf[2 * kp], kf[0], kf[1]);
        mma16816(s[t], qf[2 * kp + 1], kf[2], kf[3]);
      }
    }
    // scores to the exp2 domain, masked
    float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int t = 0; t < 4; ++t) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int h = e >> 1, key = c * kChunk + t * 8 + tid * 2 + (e & 1);
        float y = s[t][e] * p.scale_log2;
        if (p.cap_log2 != 0.f) y = tanh_exp(y) * p.cap_log2;
        if (p.slopes) y -= slope[h] * fabsf(float(pos[h] - key));
        bool see = key < lim[h];
        if (kd) see = see && __ldg(kd + (key < n ? key : 0)) == doc[h];
        s[t][e] = see ? y : -INFINITY;
        mx[h] = fmaxf(mx[h], s[t][e]);
      }
    }
    float alpha[2], mu[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 1));
      mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 2));
      const float mn = fmaxf(m[h], mx[h]);
      mu[h] = mn == -INFINITY ? 0.f : mn;  // a row that has seen nothing yet
      alpha[h] = fast_exp2(m[h] - mu[h]);
      m[h] = mn;
      l[h] *= alpha[h];
    }
    uint32_t pf[2][4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const float e0 = fast_exp2(s[t][0] - mu[0]), e1 = fast_exp2(s[t][1] - mu[0]);
      const float e2 = fast_exp2(s[t][2] - mu[1]), e3 = fast_exp2(s[t][3] - mu[1]);
      l[0] += e0 + e1;
      l[1] += e2 + e3;
      // probabilities in bf16 for the tensor core: half a step of 2^-8 each, averaged over the keys
      pf[t >> 1][(t & 1) * 2] = pack_bf16x2(e0, e1);
      pf[t >> 1][(t & 1) * 2 + 1] = pack_bf16x2(e2, e3);
    }
#pragma unroll
    for (int t = 0; t < 16; ++t) {
      o[t][0] *= alpha[0];
      o[t][1] *= alpha[0];
      o[t][2] *= alpha[1];
      o[t][3] *= alpha[1];
    }
#pragma unroll
    for (int t = 0; t < 16; ++t) {
      uint32_t vf[4];  // keys 0..31 x dims 8 t .. 8 t + 7
      const int row = lm * 8 + lr;
      ldsm4_t(vf, vs + row * 256 + ((t ^ (row & 7)) << 4));
      mma16816(o[t], pf[0], vf[0], vf[1]);
      mma16816(o[t], pf[1], vf[2], vf[3]);
    }
    __syncwarp();  // every lane is done with the slot before it is refilled
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
    l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
  }
  __syncthreads();  // the rings become the warps' partials
  float* parts = reinterpret_cast<float*>(ring);
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
  // join the warps: thread d holds column d of every row
  float* cta = parts + kWarps * kPartFloats;
  const int d = threadIdx.x;
  for (int r = 0; r < 16; ++r) {
    float mm = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, parts[w * kPartFloats + 2048 + r]);
    const float mu = mm == -INFINITY ? 0.f : mm;
    float acc = 0.f, ll = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float f = fast_exp2(parts[w * kPartFloats + 2048 + r] - mu);
      acc = fmaf(f, parts[w * kPartFloats + r * 128 + d], acc);
      ll = fmaf(f, parts[w * kPartFloats + 2064 + r], ll);
    }
    cta[r * 128 + d] = acc;
    if (d == 0) {
      cta[2048 + r] = mm;
      cta[2064 + r] = ll;
    }
  }
  if (splits > 1) cluster_sync(); else __syncthreads();
  // join the cluster: this CTA's share of the 16 rows, ranks in order
  const int r0 = rank * 16 / splits, r1 = (rank + 1) * 16 / splits;
  const uint32_t cta_addr = smem_u32(cta);
  auto peer = [&](int r, int idx) {
    float x;
    uint32_t addr = cta_addr + uint32_t(idx) * 4;
    if (splits > 1) {
      asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(addr) : "r"(addr), "r"(r));
      asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(addr) : "memory");
    } else {
      asm volatile("ld.shared.f32 %0, [%1];" : "=f"(x) : "r"(addr) : "memory");
    }
    return x;
  };
  for (int r = r0; r < r1; ++r) {
    const int row = row0 + r;
    if (row >= rows) break;
    float mm = -INFINITY;
    for (int w = 0; w < splits; ++w) mm = fmaxf(mm, peer(w, 2048 + r));
    const float mu = mm == -INFINITY ? 0.f : mm;
    float acc = 0.f, ll = 0.f;
    for (int w = 0; w < splits; ++w) {
      const float f = fast_exp2(peer(w, 2048 + r) - mu);
      acc = fmaf(f, peer(w, r * 128 + d), acc);
      ll = fmaf(f, peer(w, 2064 + r), ll);
    }
    const int i = row / p.group, g = row - i * p.group;
    const float y = ll > 0.f ? acc / ll : 0.f;
    const __nv_bfloat16 yb = __float2bfloat16_rn(y);
    p.out[b * p.o_bs + i * p.o_rs + (hk * p.group + g) * p.o_hs + d] = *reinterpret_cast<const uint16_t*>(&yb);
  }
  if (splits > 1) cluster_sync();  // no CTA leaves while its partial may be read
}

}  // namespace zi
