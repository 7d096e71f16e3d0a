// router.cu -- expert routing: scores -> top-k experts with their weights, and
// the gradient of the weights with respect to the router's logits.
//
// Per token t with logits x_e, e < E ("GLM-5.2-NVFP4" card: 256 routed experts,
// 8 per token; the gate weight of "vroomfondel/glm-5.2-reap-504B-v2-W4A4"):
//   s_e   = 1 / (1 + exp(-x_e))  or  softmax_e(x)
//   key_e = s_e + bias_e with a bias, x_e without one (both scores grow with x)
//   groups: the topk_groups of G equal runs of experts with the largest group
//           score (the largest key, or the sum of the two largest s + bias)
//   the k largest keys of the kept groups, descending, ties to the lowest index
//   w_j   = scale * s_j / (renormalize ? sum of the chosen s : 1)
// An expert whose key is -inf or NaN (a masked logit) is never chosen; missing
// choices get id -1 and weight 0.
//
// Two kernels.  k_route_few (top_k <= 16): 4 to 32 lanes per token; a lane takes
// its experts in batches of eight, sorts each batch with a fixed network and
// merges it into its running 8 or 16 largest, then the lanes' lists are merged
// pairwise by shuffles.  k_route_any, a warp per token: every other form
// (top_k > 16; softmax scores with a bias or groups ranked by two scores; group
// counts that are no power of two; and for few tokens 9 to 16 choices by score of
// up to 512 experts, and scored ones of up to 128 in ragged groups).  In both a key
// is an order-preserving integer whose low bits are replaced by the inverted expert
// index, so that one integer maximum carries the expert along and ties fall to the
// lowest index.  Where two neighbouring
// results (the largest rejected key included) agree in every bit that is left
// of the key, the token's selection runs again on the whole keys (bf16 logits
// without a bias lose no bits), as it does where a chosen key turns out to be an
// infinity or a NaN that k_route_few did not look for.
#include <cfloat>

#include "internal.h"
#include "ptx.cuh"

namespace nvfp4 {

namespace {

constexpr int kRouterWarps = 8;
constexpr uint32_t kAll = 0xffffffffu;

__device__ __forceinline__ uint32_t redux_max(uint32_t v) { return __reduce_max_sync(kAll, v); }
__device__ __forceinline__ uint32_t redux_min(uint32_t v) { return __reduce_min_sync(kAll, v); }
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
  return v;
}

// fp32 -> unsigned with the same order; 0 for what is never chosen (-inf, NaN).
__device__ __forceinline__ uint32_t order_key(float v) {
  if (!(v > -INFINITY)) return 0u;
  const uint32_t b = __float_as_uint(v + 0.0f);   // -0 counts as +0
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float sigmoid(float x) { return 1.0f / (1.0f + expf(-x)); }
// Renormalised sigmoid scores of chosen logits that are all below -20 (m: their
// largest): there s = exp(x) to within 2^-28, whose quotients exp(x - m) keep while
// s itself runs out of bits (from -87 on) and exp(-x) overflows (from -88.7 on).
// Where the largest score is 0 in fp32 all are 0.
constexpr float kTinyScores = -20.0f, kZeroScores = -103.972f;   // (2^-150 = exp(-103.972))
__device__ __forceinline__ float tiny_score(float x, float m) { return m >= kZeroScores ? expf(x - m) : 0.0f; }

__device__ __forceinline__ float load1(const float *p) { return __ldg(p); }
__device__ __forceinline__ float load1(const __nv_bfloat16 *p) {
  return __uint_as_float((uint32_t)__ldg(reinterpret_cast<const uint16_t *>(p)) << 16);
}
__device__ __forceinline__ void store1(float *p, float v) { *p = v; }
__device__ __forceinline__ void store1(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }

// +inf counts as the largest finite value (a softmax over it stays finite).
__device__ __forceinline__ float finite_top(float x) { return x > FLT_MAX ? FLT_MAX : x; }

// VEC consecutive logits (one aligned load for VEC > 1).
template <int VEC>
__device__ __forceinline__ void load_vec(const float *p, float *x) {
  if constexpr (VEC == 4) {
    const float4 v = __ldg(reinterpret_cast<const float4 *>(p));
    x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
  } else if constexpr (VEC == 2) {
    const float2 v = __ldg(reinterpret_cast<const float2 *>(p));
    x[0] = v.x; x[1] = v.y;
  } else {
    x[0] = __ldg(p);
  }
}
template <int VEC>
__device__ __forceinline__ void load_vec(const __nv_bfloat16 *p, float *x) {
  if constexpr (VEC == 8) {
    const uint4 v = __ldg(reinterpret_cast<const uint4 *>(p));
    x[0] = bf16lo(v.x); x[1] = bf16hi(v.x); x[2] = bf16lo(v.y); x[3] = bf16hi(v.y);
    x[4] = bf16lo(v.z); x[5] = bf16hi(v.z); x[6] = bf16lo(v.w); x[7] = bf16hi(v.w);
  } else if constexpr (VEC == 4) {
    const uint2 v = __ldg(reinterpret_cast<const uint2 *>(p));
    x[0] = bf16lo(v.x); x[1] = bf16hi(v.x); x[2] = bf16lo(v.y); x[3] = bf16hi(v.y);
  } else if constexpr (VEC == 2) {
    const uint32_t v = __ldg(reinterpret_cast<const uint32_t *>(p));
    x[0] = bf16lo(v); x[1] = bf16hi(v);
  } else {
    x[0] = load1(p);
  }
}

// ------------------------------------------------- selection, a warp per token --
// The k largest by k rounds of one warp-wide integer maximum (redux), which
// names the expert; removing it is one compare per key.  Issue-bound: about 835
// instructions per token at 256 experts and top 8.
// Expert of a lane's value (c, i): c * 32 * VEC + lane * VEC + i.
template <typename T, int VEC, int NCH>
__global__ void __launch_bounds__(kRouterWarps * 32) k_route_any(const RouteTopkParams p) {
  griddep_launch_dependents();
  griddep_wait();   // inputs may come from the previous kernel in the stream
  constexpr int VPL = VEC * NCH;
  extern __shared__ float sh_group[];   // groups > 1: [warps][E] values the groups are ranked by
  const int lane = threadIdx.x & 31;
  const int E = p.num_experts, k = p.top_k;
  const uint32_t imask = p.index_mask;
  const bool softmax = p.softmax != 0, whole = sizeof(T) == 2 && !p.bias;   // whole: the packed keys lose no bits
  float *gbuf = sh_group + (size_t)(threadIdx.x >> 5) * E;
  for (int64_t t = (int64_t)blockIdx.x * kRouterWarps + (threadIdx.x >> 5); t < p.tokens;
       t += (int64_t)gridDim.x * kRouterWarps) {
    const T *row = reinterpret_cast<const T *>(p.logits) + t * p.ld;
    float x[VPL];
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int e0 = c * 32 * VEC + lane * VEC;
      if (e0 < E) {
        load_vec<VEC>(row + e0, x + c * VEC);
      } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) x[c * VEC + i] = -INFINITY;
      }
    }
    // softmax statistics of the row, where the scores themselves are needed
    float row_max = 0.0f, inv_sum = 0.0f;
    if (softmax && p.need_row_sum) {
      float m = -INFINITY;
#pragma unroll
      for (int v = 0; v < VPL; ++v)
        if (x[v] > m) m = finite_top(x[v]);
      m = warp_max(m);
      float s = 0.0f;
      if (m > -INFINITY) {
#pragma unroll
        for (int v = 0; v < VPL; ++v)
          if (x[v] > -INFINITY) s += expf(finite_top(x[v]) - m);
      }
      s = warp_sum(s);
      row_max = m > -INFINITY ? m : 0.0f;
      inv_sum = s > 0.0f ? 1.0f / s : 0.0f;
    }
    // the keys: whole, and packed with the inverted index below
    uint32_t whole_key[VPL];
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const int v = c * VEC + i, e = c * 32 * VEC + lane * VEC + i;
        float key = finite_top(x[v]);
        const bool in = e < E && x[v] > -INFINITY;
        if (p.bias || p.rank_by_score) {
          float s = 0.0f;
          if (in) s = softmax ? expf(finite_top(x[v]) - row_max) * inv_sum : sigmoid(x[v]);
          if (p.bias && e < E) s += __ldg(p.bias + e);
          if (p.bias) key = in ? s : -INFINITY;
          if (p.num_groups > 1 && e < E) gbuf[e] = in && s == s ? (p.rank_by_score ? s : key) : -INFINITY;
        } else if (p.num_groups > 1 && e < E) {
          gbuf[e] = in ? key : -INFINITY;
        }
        whole_key[v] = in ? order_key(key) : 0u;
      }
    }
    if (p.num_groups > 1) {
      // lanes g*L .. g*L+L-1 scan group g for its two largest values
      __syncwarp();
      const int G = p.num_groups, per = p.group_size, L = p.group_lanes;
      const int g = lane / L, sub = lane % L;
      float t1 = -INFINITY, t2 = -INFINITY;
      if (g < G) {
        for (int i = sub; i < per; i += L) {
          const float v = gbuf[g * per + i];
          t2 = fmaxf(t2, fminf(t1, v));
          t1 = fmaxf(t1, v);
        }
      }
      for (int o = 1; o < L; o <<= 1) {
        const float o1 = __shfl_xor_sync(kAll, t1, o), o2 = __shfl_xor_sync(kAll, t2, o);
        t2 = fmaxf(fminf(t1, o1), fmaxf(t2, o2));
        t1 = fmaxf(t1, o1);
      }
      const float score = p.group_top == 2 && t2 > -INFINITY ? t1 + t2 : t1;
      int better = 0;
      for (int j = 0; j < G; ++j) {
        const float sj = __shfl_sync(kAll, score, j * L);
        better += sj > score || (sj == score && j < g);
      }
      const uint32_t keep = __ballot_sync(kAll, g < G && sub == 0 && better < p.topk_groups);
#pragma unroll
      for (int c = 0; c < NCH; ++c) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          const uint32_t e = (uint32_t)(c * 32 * VEC + lane * VEC + i);
          const uint32_t ge = (e * p.group_magic) >> 22;             // e / group_size (e < 1024)
          if (!((keep >> ((ge * (uint32_t)L) & 31u)) & 1u)) whole_key[c * VEC + i] = 0u;
        }
      }
      __syncwarp();   // the next token's values overwrite the buffer
    }
    uint32_t key[VPL];
    uint32_t lmax = 0;
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const int v = c * VEC + i;
        const uint32_t e = (uint32_t)(c * 32 * VEC + lane * VEC + i);
        key[v] = whole_key[v] ? (whole_key[v] & ~imask) | (imask - e) : 0u;
        lmax = max(lmax, key[v]);
      }
    }
    int id = -1;
    uint32_t prev = 0;
    bool close = false;        // two neighbours agree in the bits that are left
    for (int j = 0; j <= k; ++j) {
      const uint32_t m = redux_max(lmax);
      if (m == 0u) break;
      if (j > 0) close |= ((m ^ prev) & ~imask) == 0u;
      prev = m;
      if (j == k) break;
      if (lane == j) id = (int)(imask - (m & imask));
      lmax = 0;
#pragma unroll
      for (int v = 0; v < VPL; ++v) {
        key[v] = key[v] == m ? 0u : key[v];
        lmax = max(lmax, key[v]);
      }
    }
    if (close && !whole) {
      id = -1;
      for (int j = 0; j < k; ++j) {
        uint32_t lm = 0;
#pragma unroll
        for (int v = 0; v < VPL; ++v) lm = max(lm, whole_key[v]);
        const uint32_t m = redux_max(lm);
        if (m == 0u) break;
        uint32_t cand = 0xffffffffu;
#pragma unroll
        for (int c = NCH - 1; c >= 0; --c) {
#pragma unroll
          for (int i = VEC - 1; i >= 0; --i)
            if (whole_key[c * VEC + i] == m) cand = (uint32_t)(c * 32 * VEC + lane * VEC + i);
        }
        const uint32_t e = redux_min(cand);
        if (lane == j) id = (int)e;
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
#pragma unroll
          for (int i = 0; i < VEC; ++i)
            if ((uint32_t)(c * 32 * VEC + lane * VEC + i) == e) whole_key[c * VEC + i] = 0u;
        }
      }
    }
    // the weights, from the chosen experts' logits (lane j: choice j)
    const float xs = id >= 0 ? load1(row + id) : -INFINITY;
    float w = 0.0f;
    if (softmax) {
      if (p.renormalize) {
        const float m = warp_max(finite_top(xs));
        w = id >= 0 ? expf(finite_top(xs) - m) : 0.0f;
        const float s = warp_sum(w);
        w = s > 0.0f ? w / s : 0.0f;
      } else if (id >= 0) {
        w = expf(finite_top(xs) - row_max) * inv_sum;
      }
    } else {
      const float m = p.renormalize ? warp_max(xs) : 0.0f;
      if (id >= 0) w = m < kTinyScores ? tiny_score(xs, m) : sigmoid(xs);
      if (p.renormalize) {
        const float s = warp_sum(w);
        w = s > 0.0f ? w / s : 0.0f;
      }
    }
    if (lane < k) {
      p.expert_ids[t * k + lane] = id;
      p.weights[t * k + lane] = w * p.scale;
    }
  }
}

// ----------------------------------------- selection, up to 16 experts per token --
// Descending order of keys a, b.
__device__ __forceinline__ void cex(uint32_t &a, uint32_t &b) {
  const uint32_t hi = max(a, b);
  b = min(a, b);
  a = hi;
}
// A 19-comparator sorting network for eight keys (its six layers; every
// 0/1 input is sorted, which proves it for all).
__device__ __forceinline__ void sort8(uint32_t (&v)[8]) {
  cex(v[0], v[2]); cex(v[1], v[3]); cex(v[4], v[6]); cex(v[5], v[7]);
  cex(v[0], v[4]); cex(v[1], v[5]); cex(v[2], v[6]); cex(v[3], v[7]);
  cex(v[0], v[1]); cex(v[2], v[3]); cex(v[4], v[5]); cex(v[6], v[7]);
  cex(v[2], v[4]); cex(v[3], v[5]);
  cex(v[1], v[4]); cex(v[3], v[6]);
  cex(v[1], v[2]); cex(v[3], v[4]); cex(v[5], v[6]);
}
// run (R sorted keys) <- the R largest of run and v (V <= R sorted ones): the
// elementwise maxima of one and the other reversed (zeros behind v's V) are
// them, as a bitonic sequence.  kRest: rest <- the largest key that ever lost.
template <bool kRest, int R, int V>
__device__ __forceinline__ void merge(uint32_t (&run)[R], const uint32_t (&v)[V], uint32_t &rest) {
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const uint32_t a = run[R - V + i], b = v[V - 1 - i];
    run[R - V + i] = max(a, b);
    if (kRest) rest = max(rest, min(a, b));
  }
#pragma unroll
  for (int o = R / 2; o > 0; o >>= 1) {
#pragma unroll
    for (int i = 0; i < R; ++i)
      if (!(i & o)) cex(run[i], run[i + o]);
  }
}

// Eight consecutive logits: two or one 16-byte loads, or (kVec false) the n
// first of them, -inf behind.
template <typename T, bool kVec>
__device__ __forceinline__ void load_eight(const T *p, int n, float (&x)[8]) {
  if constexpr (kVec) {
    constexpr int V = 16 / (int)sizeof(T);
#pragma unroll
    for (int i = 0; i < 8; i += V) load_vec<V>(p + i, x + i);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = i < n ? load1(p + i) : -INFINITY;
  }
}

// The packed keys of eight experts from e0 (a multiple of 8) on, keys that are
// the logits, without a look at infinities and NaNs: positive ones and +inf
// land at or above 0xFF800000, -inf and the negative ones below 0x00800000,
// where the caller finds them if they were chosen.
__device__ __forceinline__ void plain_keys(const float *p, int e0, uint32_t imask, uint32_t (&v)[8], float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 8; i += 4) load_vec<4>(p + i, x + i);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t b = __float_as_uint(x[i] + 0.0f);                      // -0 counts as +0
    const uint32_t u = b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
    v[i] = (u & ~imask) | (imask - (uint32_t)(e0 + i));
  }
}
// bf16: two experts per word until the index comes in below their 16 bits.
__device__ __forceinline__ void plain_keys(const __nv_bfloat16 *p, int e0, uint32_t imask, uint32_t (&v)[8],
                                           float (&x)[8]) {
  const uint4 q = __ldg(reinterpret_cast<const uint4 *>(p));
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
  const uint32_t index = (imask - (uint32_t)e0) * 0x00010001u - 0x00010000u;   // low half: expert e0, high: e0 + 1
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t b;                                                           // x * 1 + 0: -0 becomes +0
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(b) : "r"(w[j]), "r"(0x3F803F80u), "r"(0u));
    uint32_t sign;                                                        // each half's sign, 16 times
    asm("prmt.b32 %0, %1, %2, 0xBB99;" : "=r"(sign) : "r"(b), "r"(0u));
    const uint32_t u = b ^ (sign | 0x80008000u);
    const uint32_t at = index - 0x00020002u * j;
    v[2 * j] = __byte_perm(u, at, 0x1054);
    v[2 * j + 1] = __byte_perm(u, at, 0x3276);
    x[2 * j] = bf16lo(w[j]);
    x[2 * j + 1] = bf16hi(w[j]);
  }
}

// The key and the value that groups are ranked by, of expert e.
template <bool kScored>
__device__ __forceinline__ uint32_t route_key(const float *bias, int e, float x, float &gval) {
  bool in = x > -INFINITY;
  float key, s = x;
  if (kScored) s = sigmoid(x);
  if (kScored && bias) {
    s += __ldg(bias + e);
    key = s;
    in = in && key > -INFINITY;
  } else {
    key = fminf(x, FLT_MAX);         // +inf counts as the largest finite value (a NaN is not in)
  }
  gval = in ? s : -INFINITY;         // (kScored without a bias: only where groups are ranked by scores)
  const uint32_t b = __float_as_uint(key + 0.0f);                       // -0 counts as +0
  const uint32_t u = b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
  return in ? u : 0u;
}

// The exact selection of one token by a whole warp, from choice `from` on: each
// round the largest (key, lowest index) below the previous one's, last and
// last_e (~0 and -1: none).  Lane j >= from returns choice j.  (Its arguments go
// by value: the whole struct by reference cost every caller a copy on the stack.)
template <typename T, bool kScored>
__device__ __noinline__ int route_exact(const T *row, const float *bias, int num_experts, int top_k,
                                        uint32_t group_magic, uint32_t keep, int from, uint32_t last, int last_e) {
  const int lane = threadIdx.x & 31;
  int id = -1;
  for (int j = from; j < top_k; ++j) {
    uint32_t best = 0u;
    int best_e = 0;
    for (int e = lane; e < num_experts; e += 32) {
      if (!((keep >> ((uint32_t)e * group_magic >> 22)) & 1u)) continue;
      float g;
      const uint32_t u = route_key<kScored>(bias, e, load1(row + e), g);
      if ((u < last || (u == last && e > last_e)) && u > best) {
        best = u;
        best_e = e;
      }
    }
    const uint32_t m = redux_max(best);
    if (m == 0u) break;
    last = m;
    last_e = (int)redux_min(best == m ? (uint32_t)best_e : 0xffffffffu);
    if (lane == j) id = last_e;
  }
  return id;
}

// Per eight keys the network takes 19 comparators, the merge 8 maxima and 12
// comparators: 70 integer minima and maxima, which run at half rate and bound the
// kernel (ALU pipe 70-85% busy): 65521 tokens, 256 experts, bf16, top 8 in 17.6 us
// (37.7 MB, 2.1 TB/s); the one-warp-per-token kernel above took 69 us.
// R = 16 (top_k 9 to 16): a merge of 8 maxima and 32 comparators; 65521 tokens, 256
// experts, bf16, top 10 in 29.7 us (the one-warp-per-token kernel: 73 us).
// L lanes per token.  kScored: keys or group values are sigmoid scores; kVec:
// a lane's eight experts are whole 16-byte vectors.  With groups L / G lanes
// share a group and take a run of its experts each (the last ones a shorter one
// or none); without, the lanes' batches of eight interleave.
template <typename T, int L, int R, bool kScored, bool kVec>
__global__ void __launch_bounds__(kRouterWarps * 32) k_route_few(const RouteTopkParams p) {
  griddep_launch_dependents();
  griddep_wait();   // inputs may come from the previous kernel in the stream
  constexpr bool kRest = kScored || sizeof(T) == 4;    // packed keys may lose bits
  constexpr bool kPlain = !kScored && kVec;            // keys without a look at infinities and NaNs
  constexpr int kTok = 32 / L;                         // tokens per warp
  const int lane = threadIdx.x & 31, sub = lane % L;
  const int E = p.num_experts, k = p.top_k;
  const uint32_t imask = p.index_mask;
  const bool grouped = p.num_groups > 1;
  int first = sub * 8, end = E;
  const int step = grouped ? 8 : 8 * L;
  if (grouped) {
    const int shift = __ffs(L) - __ffs(p.num_groups), lanes = 1 << shift, g = sub >> shift;
    const int run = (p.group_size + lanes - 1) >> shift;
    end = (g + 1) * p.group_size;
    first = min(g * p.group_size + (sub & (lanes - 1)) * run, end);
    end = min(first + run, end);
  }
  const int64_t stride = (int64_t)gridDim.x * kRouterWarps * kTok;
  for (int64_t t0 = ((int64_t)blockIdx.x * kRouterWarps + (threadIdx.x >> 5)) * kTok; t0 < p.tokens; t0 += stride) {
    const int64_t t = t0 + lane / L;
    const bool live = t < p.tokens;
    const T *row = reinterpret_cast<const T *>(p.logits) + (live ? t : t0) * p.ld;
    uint32_t run[R], rest = 0u;
#pragma unroll
    for (int i = 0; i < R; ++i) run[i] = 0u;
    float t1 = -INFINITY, t2 = -INFINITY, row_max = -INFINITY;
    for (int e0 = first; e0 < end; e0 += step) {
      float x[8];
      uint32_t v[8];
      if constexpr (kPlain) {
        plain_keys(row + e0, e0, imask, v, x);
        if (grouped) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float g = x[i] > -INFINITY ? x[i] : -INFINITY;
            t2 = fmaxf(t2, fminf(t1, g));
            t1 = fmaxf(t1, g);
          }
        }
        if (p.need_row_sum) {
#pragma unroll
          for (int i = 0; i < 8; ++i) row_max = fmaxf(row_max, x[i]);         // (fmaxf passes over NaN)
          row_max = finite_top(row_max);
        }
        sort8(v);
        merge<kRest>(run, v, rest);
        continue;
      }
      load_eight<T, kVec>(row + e0, end - e0, x);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int e = kVec ? e0 + i : min(e0 + i, E - 1);
        float g;
        const uint32_t u = route_key<kScored>(p.bias, e, x[i], g);
        v[i] = u ? (u & ~imask) | (imask - (uint32_t)e) : 0u;
        if (grouped) {
          t2 = fmaxf(t2, fminf(t1, g));
          t1 = fmaxf(t1, g);
        }
        if (!kScored && p.need_row_sum) row_max = fmaxf(row_max, finite_top(x[i]));   // (fmaxf passes over NaN)
      }
      sort8(v);
      merge<kRest>(run, v, rest);
    }
    uint32_t keep = 0xffffffffu;       // groups that stay, bit g
    if (grouped) {
      const int G = p.num_groups, per = 1 << (__ffs(L) - __ffs(G));       // lanes per group
      for (int o = 1; o < per; o <<= 1) {
        const float o1 = __shfl_xor_sync(kAll, t1, o), o2 = __shfl_xor_sync(kAll, t2, o);
        t2 = fmaxf(fminf(t1, o1), fmaxf(t2, o2));
        t1 = fmaxf(t1, o1);
      }
      // (logits rank groups by their largest alone: a sum of two is of scores)
      const float score = !kScored ? finite_top(t1) : p.group_top == 2 && t2 > -INFINITY ? t1 + t2 : t1;
      const int g = sub >> (__ffs(L) - __ffs(G));
      int better = 0;
      keep = 0u;
      for (int j = 0; j < G; ++j) {
        const float sj = __shfl_sync(kAll, score, (lane - sub) + j * per);
        better += sj > score || (sj == score && j < g);
      }
      const uint32_t votes = __ballot_sync(kAll, better < p.topk_groups);
      for (int j = 0; j < G; ++j) keep |= ((votes >> ((lane - sub) + j * per)) & 1u) << j;
      if (better >= p.topk_groups) {
        rest = 0u;
#pragma unroll
        for (int i = 0; i < R; ++i) run[i] = 0u;
      }
    }
#pragma unroll
    for (int o = 1; o < L; o <<= 1) {
      uint32_t v[R];
#pragma unroll
      for (int i = 0; i < R; ++i) v[i] = __shfl_xor_sync(kAll, run[i], o);
      if (kRest) rest = max(rest, __shfl_xor_sync(kAll, rest, o));
      merge<kRest>(run, v, rest);
    }
    // this lane's choices: slots sub, sub + L, ... (two for L < R)
    constexpr int kSlots = L >= R ? 1 : R / L;
    int id[kSlots];
#pragma unroll
    for (int q = 0; q < kSlots; ++q) {
      uint32_t m = 0u;
#pragma unroll
      for (int i = 0; i < R; ++i)
        if (i == sub + q * L) m = run[i];
      id[q] = m && sub + q * L < k ? (int)(imask - (m & imask)) : -1;
    }
    if constexpr (kRest || kPlain) {
      bool close = false, redo = kPlain && run[0] >= 0xFF800000u;
      int sure = k;                    // choices that no key outside the list can take
#pragma unroll
      for (int i = R - 1; i >= 0; --i) {
        if (kPlain) redo |= i < k && run[i] < 0x00800000u;
        // neighbours that agree in the bits that are left
        if (kRest) {
          if (i < k && rest && ((run[i] ^ rest) & ~imask) == 0u) sure = i;
          const uint32_t below = i < R - 1 ? run[i < R - 1 ? i + 1 : i] : 0u;
          close |= i < k && below && ((run[i] ^ below) & ~imask) == 0u;
        }
      }
      uint32_t whole[kSlots];          // of this lane's slots, once they are known
      if (kRest && __any_sync(kAll, close || sure < k)) {
        // the list in the order of its whole keys
        int e[kSlots], rank[kSlots];
#pragma unroll
        for (int q = 0; q < kSlots; ++q) {
          uint32_t m = 0u;
#pragma unroll
          for (int i = 0; i < R; ++i)
            if (i == sub + q * L) m = run[i];
          float g;
          e[q] = m ? (int)(imask - (m & imask)) : E;
          whole[q] = m ? route_key<kScored>(p.bias, e[q], load1(row + e[q]), g) : 0u;
          rank[q] = 0;
        }
#pragma unroll
        for (int j = 0; j < R; ++j) {
          const uint32_t wj = __shfl_sync(kAll, whole[j / L], lane - sub + j % L);
          const int ej = __shfl_sync(kAll, e[j / L], lane - sub + j % L);
#pragma unroll
          for (int q = 0; q < kSlots; ++q)
            rank[q] += wj > whole[q] || (wj == whole[q] && (ej < e[q] || (ej == e[q] && j < sub + q * L)));
        }
        uint32_t sorted[kSlots];
#pragma unroll
        for (int j = 0; j < R; ++j) {
          const uint32_t wj = __shfl_sync(kAll, whole[j / L], lane - sub + j % L);
          const int ej = __shfl_sync(kAll, e[j / L], lane - sub + j % L);
          const int rj = __shfl_sync(kAll, rank[j / L], lane - sub + j % L);
#pragma unroll
          for (int q = 0; q < kSlots; ++q) {
            if (rj == sub + q * L) {
              sorted[q] = wj;
              id[q] = wj && rj < k ? ej : -1;
            }
          }
        }
#pragma unroll
        for (int q = 0; q < kSlots; ++q) whole[q] = sorted[q];
      }
      uint32_t again = __ballot_sync(kAll, (redo || sure < k) && live && sub == 0);
      while (again) {
        const int src = __ffs(again) - 1;            // the token's first lane
        again &= again - 1;
        const T *r = reinterpret_cast<const T *>(p.logits) + (t0 + src / L) * p.ld;
        const int from = kRest ? __shfl_sync(kAll, redo ? 0 : sure, src) : 0;
        uint32_t last = 0xffffffffu;
        int last_e = -1;
        if (kRest && from > 0) {
#pragma unroll
          for (int q = 0; q < kSlots; ++q) {
            const uint32_t lw = __shfl_sync(kAll, whole[q], src + (from - 1) % L);
            const int le = __shfl_sync(kAll, id[q], src + (from - 1) % L);
            if ((from - 1) / L == q) {
              last = lw;
              last_e = le;
            }
          }
        }
        const uint32_t groups = __shfl_sync(kAll, keep, src);
        const int e = route_exact<T, kScored>(r, p.bias, E, k, p.group_magic, groups, from, last, last_e);
#pragma unroll
        for (int q = 0; q < kSlots; ++q) {
          const int v = __shfl_sync(kAll, e, (sub + q * L) & 31);
          if (lane - sub == src && sub + q * L >= from) id[q] = sub + q * L < k ? v : -1;
        }
      }
    }
    const auto sum_tok = [](float v) {
#pragma unroll
      for (int o = 1; o < L; o <<= 1) v += __shfl_xor_sync(kAll, v, o);
      return v;
    };
    const auto max_tok = [](float v) {
#pragma unroll
      for (int o = 1; o < L; o <<= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
      return v;
    };
    float w[kSlots], total = 0.0f;
    if (p.softmax) {
      float xs[kSlots], m = -INFINITY;
#pragma unroll
      for (int q = 0; q < kSlots; ++q) {
        xs[q] = id[q] >= 0 ? finite_top(load1(row + id[q])) : -INFINITY;
        m = fmaxf(m, xs[q]);
      }
      if (p.need_row_sum) m = row_max;
      m = max_tok(m);
      if (!(m > -INFINITY)) m = 0.0f;
      if (p.need_row_sum) {            // the scores' denominator: the whole row
        for (int e0 = first; e0 < end; e0 += step) {
          float x[8];
          load_eight<T, kVec>(row + e0, end - e0, x);
          // (exp2 approximations: the terms that count are within a few of m)
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (x[i] > -INFINITY) total += __expf(finite_top(x[i]) - m);
        }
      }
#pragma unroll
      for (int q = 0; q < kSlots; ++q) {
        w[q] = id[q] >= 0 ? expf(xs[q] - m) : 0.0f;
        if (!p.need_row_sum) total += w[q];
      }
    } else {
      float xs[kSlots], m = -INFINITY;
#pragma unroll
      for (int q = 0; q < kSlots; ++q) {
        xs[q] = id[q] >= 0 ? load1(row + id[q]) : -INFINITY;
        m = fmaxf(m, xs[q]);
      }
      m = p.renormalize ? max_tok(m) : 0.0f;
#pragma unroll
      for (int q = 0; q < kSlots; ++q) {
        w[q] = id[q] < 0 ? 0.0f : m < kTinyScores ? tiny_score(xs[q], m) : sigmoid(xs[q]);
        total += w[q];
      }
    }
    total = sum_tok(total);
    const bool divide = p.softmax || p.renormalize;
#pragma unroll
    for (int q = 0; q < kSlots; ++q) {
      const int slot = sub + q * L;
      if (divide) w[q] = total > 0.0f ? w[q] / total : 0.0f;
      if (live && slot < k) {
        p.expert_ids[t * k + slot] = id[q];
        p.weights[t * k + slot] = w[q] * p.scale;
      }
    }
  }
}

// ----------------------------------------------------------------- gradient --
// With d_j = scale * grad_w_j (0 for an id outside [0, E)) and the choice held fixed:
//   sigmoid:  ds_j = renormalize ? (d_j - sum_i d_i w_i) / S : d_j,  w_i = s_i / S,  S = sum_i s_i
//             dx_j = ds_j s_j (1 - s_j) on the chosen experts, 0 elsewhere
//   softmax, renormalized: the weights are the softmax over the chosen logits:
//             dx_j = w_j (d_j - sum_i d_i w_i) on the chosen experts, 0 elsewhere
//   softmax:  dx_e = p_e (d_e - sum_j d_j p_j) for every expert
// L lanes per token (8, or a warp where top_k > 8 or E > 256).  The row is
// written whole -- zeros, in 16-byte vectors where it allows them (kVec), or p_e
// times minus the dot product (kDense) -- and the chosen experts' elements over
// it.  HBM-bound: that write and, with kDense, the read of the logits.  This
// kernel serves the sparse forms, and the dense one for rows that are not whole
// 16-byte vectors, an element at a time.
// The exponentials of the dense form are exp2 approximations: with |x - max| <
// 64 their relative error stays below 2^-17 (most of it the rounding of the
// exponent's argument, which is why it is small where the term is large).
template <typename T, int L, bool kVec, bool kDense>
__global__ void __launch_bounds__(kRouterWarps * 32) k_route_topk_backward(const RouteGradParams p) {
  griddep_launch_dependents();
  griddep_wait();   // inputs may come from the previous kernel in the stream
  constexpr int VEC = kVec ? 16 / (int)sizeof(T) : 1;
  constexpr int kTok = 32 / L;
  const int lane = threadIdx.x & 31, sub = lane % L;
  const int E = p.num_experts, k = p.top_k;
  const auto sum_tok = [](float v) {
#pragma unroll
    for (int o = 1; o < L; o <<= 1) v += __shfl_xor_sync(kAll, v, o);
    return v;
  };
  const auto max_tok = [](float v) {
#pragma unroll
    for (int o = 1; o < L; o <<= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
    return v;
  };
  const int64_t stride = (int64_t)gridDim.x * kRouterWarps * kTok;
  for (int64_t t0 = ((int64_t)blockIdx.x * kRouterWarps + (threadIdx.x >> 5)) * kTok; t0 < p.tokens; t0 += stride) {
    const int64_t t = t0 + lane / L;
    const bool live = t < p.tokens;
    const T *row = reinterpret_cast<const T *>(p.logits) + (live ? t : t0) * p.ld;
    T *out = reinterpret_cast<T *>(p.grad_logits) + (live ? t : t0) * p.ld_grad;
    int id = live && sub < k ? __ldg(p.expert_ids + t * k + sub) : -1;
    if (id >= E) id = -1;
    const float d = id >= 0 ? __ldg(p.grad_weights + t * k + sub) * p.scale : 0.0f;
    const float xs = id >= 0 ? load1(row + id) : -INFINITY;
    float g = 0.0f;                    // of the chosen expert
    if constexpr (kDense) {
      // running maximum and sum of the lane's part of the row, then of the token
      static_assert(!kVec, "rows of whole vectors take k_route_softmax_backward");
      float m = -INFINITY, s = 0.0f;
      for (int e = sub; e < E; e += L) {
        const float x = finite_top(load1(row + e));
        const float top = fmaxf(m, x);                        // (fmaxf passes over NaN)
        if (top > -INFINITY) {
          s *= __expf(m - top);
          m = top;
          if (x > -INFINITY) s += __expf(x - m);
        }
      }
      const float top = max_tok(m);
      const float mt = top > -INFINITY ? top : 0.0f;          // an empty row: every p is 0
      s = sum_tok(m > -INFINITY ? s * __expf(m - mt) : 0.0f);
      const float inv = s > 0.0f ? 1.0f / s : 0.0f;
      const float ps = xs > -INFINITY ? __expf(finite_top(xs) - mt) * inv : 0.0f;
      const float dot = sum_tok(d * ps);
      g = ps * (d - dot);
      if (live) {
        const float c = -dot * inv;
        for (int e = sub; e < E; e += L) {
          const float x = load1(row + e);
          store1(out + e, x > -INFINITY ? __expf(finite_top(x) - mt) * c : 0.0f);
        }
      }
    } else {
      if (live) {
        for (int e = sub * VEC; e < E; e += L * VEC) {
          if constexpr (kVec)
            *reinterpret_cast<uint4 *>(out + e) = make_uint4(0, 0, 0, 0);
          else
            store1(out + e, 0.0f);
        }
      }
      if (p.softmax) {                       // renormalized
        const float m = max_tok(finite_top(xs));
        const float e = xs > -INFINITY ? expf(finite_top(xs) - m) : 0.0f;
        const float s = sum_tok(e);
        const float w = s > 0.0f ? e / s : 0.0f;
        const float c = sum_tok(d * w);
        g = w * (d - c);
      } else {
        // s (1 - s) from exp(-|x|): 1 - s would cancel for large x
        const float a = expf(-fabsf(xs));
        const float slope = a / ((1.0f + a) * (1.0f + a));
        if (p.renormalize) {
          // slope / S <= 1 whatever the size of S: 1 / S alone may overflow
          const float m = max_tok(xs);
          const bool tiny = m < kTinyScores;       // slope = s there
          const float s = id < 0 ? 0.0f : tiny ? tiny_score(xs, m) : sigmoid(xs);
          const float S = sum_tok(s);
          const float c = sum_tok(S > 0.0f ? d * (s / S) : 0.0f);
          g = id >= 0 && S > 0.0f ? (d - c) * ((tiny ? s : slope) / S) : 0.0f;
        } else {
          g = id >= 0 ? d * slope : 0.0f;
        }
      }
    }
    __syncwarp();      // the row's stores come before the chosen experts'
    if (id >= 0) store1(out + id, g);
  }
}

// The dense softmax form with the row in registers: 32 / VEC vectors per lane
// (L = 8: up to 256 experts, L = 32: up to 1024), one exponential per element.
// 65521 tokens, 160 experts, bf16: 10.0 us of 45.1 MB = 4.5 TB/s (18 us when the
// row was read twice, 13.7 us with the chosen logits' loads, which wait for the
// ids, issued before the row's); bound by load latency.
// The first attempt takes every logit for finite and the maximum for small
// enough that its product with log2(e) keeps its fraction: rounding that product
// scales every term of the row by the same 2^r.  Up to 1024 terms, the largest
// of them 2^r, sum to between 2^r and 2^(r + 10), so a sum in [1/2, 2048] bounds r
// by 11.  A row with any other sum (a maximum that is infinite or beyond about
// 1e8, a NaN) sends its warp through a second attempt, which takes x - m before
// the product, masks -inf and NaN and takes +inf for the largest fp32.
template <typename T, int L>
__global__ void __launch_bounds__(kRouterWarps * 32, 5) k_route_softmax_backward(const RouteGradParams p) {
  griddep_launch_dependents();
  griddep_wait();   // inputs may come from the previous kernel in the stream
  constexpr int VEC = 16 / (int)sizeof(T), NV = 32 / VEC, kTok = 32 / L;
  constexpr float kLog2e = 1.44269504f;
  const int lane = threadIdx.x & 31, sub = lane % L;
  const int E = p.num_experts, k = p.top_k;
  const auto sum_tok = [](float v) {
#pragma unroll
    for (int o = 1; o < L; o <<= 1) v += __shfl_xor_sync(kAll, v, o);
    return v;
  };
  const int64_t stride = (int64_t)gridDim.x * kRouterWarps * kTok;
  for (int64_t t0 = ((int64_t)blockIdx.x * kRouterWarps + (threadIdx.x >> 5)) * kTok; t0 < p.tokens; t0 += stride) {
    const int64_t t = t0 + lane / L;
    const bool live = t < p.tokens;
    const T *row = reinterpret_cast<const T *>(p.logits) + (live ? t : t0) * p.ld;
    T *out = reinterpret_cast<T *>(p.grad_logits) + (live ? t : t0) * p.ld_grad;
    // every load is issued before the first use: the ids and their gradients,
    // the row, then (the one that depends on another) the chosen logits
    const bool slot = live && sub < k;
    int id = slot ? __ldg(p.expert_ids + t * k + sub) : -1;
    float d = slot ? __ldg(p.grad_weights + t * k + sub) * p.scale : 0.0f;
    float x[NV][VEC], m, s, ps;
    const auto load_row = [&]() {
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int e = (v * L + sub) * VEC;
#pragma unroll
        for (int i = 0; i < VEC; ++i) x[v][i] = -INFINITY;
        if (e < E) load_vec<VEC>(row + e, x[v]);
      }
    };
    load_row();
    if (id < 0 || id >= E) {
      id = -1;
      d = 0.0f;
    }
    const float xs = id >= 0 ? load1(row + id) : -INFINITY;
    for (int attempt = 0;; ++attempt) {
      if (attempt) load_row();
      m = -INFINITY;
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        if (v * L * VEC >= E) continue;
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          if (attempt) x[v][i] = x[v][i] > -INFINITY ? finite_top(x[v][i]) : -INFINITY;
          m = fmaxf(m, x[v][i]);
        }
      }
#pragma unroll
      for (int o = 1; o < L; o <<= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, o));
      if (attempt && !(m > -INFINITY)) m = 0.0f;         // an empty row: every p is 0
      const float shift = m * kLog2e;
      s = 0.0f;
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        if (v * L * VEC >= E) continue;
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          x[v][i] = attempt ? __expf(x[v][i] - m) : exp2_approx(fmaf(x[v][i], kLog2e, -shift));
          s += x[v][i];
        }
      }
      s = sum_tok(s);
      ps = attempt ? (xs > -INFINITY ? __expf(finite_top(xs) - m) : 0.0f) : exp2_approx(fmaf(xs, kLog2e, -shift));
      if (attempt || __all_sync(kAll, s >= 0.5f && s <= 2048.0f)) break;   // (a NaN compares false)
    }
    const float inv = s > 0.0f ? 1.0f / s : 0.0f;
    ps *= inv;
    const float dot = sum_tok(d * ps);
    const float c = -dot * inv;
    if (live) {
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int e = (v * L + sub) * VEC;
        if (e >= E) continue;
        if constexpr (VEC == 8) {
          uint32_t o[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x[v][2 * i] * c, x[v][2 * i + 1] * c);
            o[i] = *reinterpret_cast<const uint32_t *>(&h);
          }
          *reinterpret_cast<uint4 *>(out + e) = make_uint4(o[0], o[1], o[2], o[3]);
        } else {
          *reinterpret_cast<float4 *>(out + e) =
              make_float4(x[v][0] * c, x[v][1] * c, x[v][2] * c, x[v][3] * c);
        }
      }
    }
    __syncwarp();      // the row's stores come before the chosen experts'
    if (id >= 0) store1(out + id, ps * (d - dot));
  }
}

template <typename T, int VEC, int NCH>
cudaError_t launch_topk(const RouteTopkParams &p, int num_sms, cudaStream_t st) {
  const size_t smem = p.num_groups > 1 ? (size_t)kRouterWarps * p.num_experts * 4 : 0;   // <= 32 KB
  const int64_t ctas = std::min<int64_t>((p.tokens + kRouterWarps - 1) / kRouterWarps, (int64_t)num_sms * 8);
  return launch_pdl(k_route_any<T, VEC, NCH>, dim3((unsigned)ctas), dim3(kRouterWarps * 32), smem, st, p);
}

template <typename T, int L, int R, bool kScored>
cudaError_t launch_few(const RouteTopkParams &p, bool vec, int num_sms, cudaStream_t st) {
  const int64_t per_cta = (int64_t)kRouterWarps * (32 / L);
  const int64_t ctas = std::min<int64_t>((p.tokens + per_cta - 1) / per_cta, (int64_t)num_sms * 64);
  const dim3 grid((unsigned)ctas), block(kRouterWarps * 32);
  return vec ? launch_pdl(k_route_few<T, L, R, kScored, true>, grid, block, 0, st, p)
             : launch_pdl(k_route_few<T, L, R, kScored, false>, grid, block, 0, st, p);
}
// Lanes per token: enough warps for the device with as few lanes as that takes --
// every halving of L saves a merge and its shuffles per token -- but at least eight
// experts per lane; with groups, whole lanes per group.  Enough is 8 to 32 warps per
// SM, in step with the experts, whose batches a lane takes one after the other: top
// 8 of 160 experts, 8192 tokens, bf16 4.6 us with 8 warps and 6.2 with 16; of 1000,
// 32768 tokens 29.1 with 32, 40.8 with 16; of 256, 16384 tokens fp32 with a bias 17.6 with 16,
// 20.7 with 8, 18.1 with 32.  4 with lists of 16, whose merges cost more: 2048 tokens,
// 256 experts, top 10 4.0 us, with 2 4.8, with 8 5.8.
template <typename T, int R, bool kScored>
cudaError_t pick_few(const RouteTopkParams &p, int num_sms, cudaStream_t st) {
  const int E = p.num_experts, G = p.num_groups;
  int L = 32;
  const int64_t enough = (int64_t)num_sms * (R == 8 ? std::min(std::max(E / 16, 8), 32) : 4) * 32;
  while (L > R / 2 && (L > G || G == 1) && (p.tokens * (L / 2) >= enough || E < 8 * L)) L /= 2;
  L = std::max(L, G);
  const bool vec = E % 8 == 0 && (G == 1 || E % (8 * L) == 0) && p.ld * sizeof(T) % 16 == 0 &&
                   reinterpret_cast<uintptr_t>(p.logits) % 16 == 0;
  if constexpr (R == 8)
    if (L == 4) return launch_few<T, 4, R, kScored>(p, vec, num_sms, st);
  switch (L) {
    case 8: return launch_few<T, 8, R, kScored>(p, vec, num_sms, st);
    case 16: return launch_few<T, 16, R, kScored>(p, vec, num_sms, st);
    default: return launch_few<T, 32, R, kScored>(p, vec, num_sms, st);
  }
}
// The forms that k_route_few takes: up to 16 choices; keys that need no row
// statistics; a power of two of groups, up to 32 (whole lanes for each).  Lists
// of 16 scored keys only for many tokens or more than 512 experts: few tokens wait
// longer for the few lanes' scores than for a warp's (fp32, bias, top 10, against the
// other kernel: 4096 tokens of 256 experts 12.1 and 9.5 us, of 512 18.2 and 18.2, of 1000
// 29.3 and 46.2; 16384 tokens of 256 20.9 and 24.7).  Few tokens of up to 128 experts
// by score in groups that are no whole batches of eight neither: 64 tokens of 44 in 4
// groups 7.3 against 4.4 us, 512 of 100 in 4 6.5 and 5.0; 8192 of 100 8.9 and 10.8, 64 of
// 264 in 8 6.8 and 8.5.
bool takes_few(const RouteTopkParams &p, bool scored, int num_sms) {
  if (p.top_k > 16 || (p.softmax && (p.bias || p.rank_by_score))) return false;
  if (p.top_k > 8 && scored && p.num_experts <= 512 && p.tokens < (int64_t)num_sms * 64) return false;
  const int G = p.num_groups;
  if (scored && G > 1 && p.num_experts <= 128 && p.group_size % 8 != 0 && p.tokens < (int64_t)num_sms * 16)
    return false;
  return G <= 32 && (G & (G - 1)) == 0;
}

// Values per lane by the number of experts; vector loads where the rows allow
// them (every row starts on the vector's size and E is a multiple of it).
template <typename T>
cudaError_t pick_topk(const RouteTopkParams &p, int num_sms, cudaStream_t st) {
  const int E = p.num_experts;
  const bool scored = !p.softmax && (p.bias || p.rank_by_score);
  if (takes_few(p, scored, num_sms)) {
    if (p.top_k <= 8) return scored ? pick_few<T, 8, true>(p, num_sms, st) : pick_few<T, 8, false>(p, num_sms, st);
    return scored ? pick_few<T, 16, true>(p, num_sms, st) : pick_few<T, 16, false>(p, num_sms, st);
  }
  const auto vec_ok = [&](int vec) {
    return E % vec == 0 && p.ld % vec == 0 && reinterpret_cast<uintptr_t>(p.logits) % (vec * sizeof(T)) == 0;
  };
  if (E <= 64 && vec_ok(2)) return launch_topk<T, 2, 1>(p, num_sms, st);
  if (E <= 128 && vec_ok(4)) return launch_topk<T, 4, 1>(p, num_sms, st);
  if constexpr (sizeof(T) == 2) {
    if (E <= 256 && vec_ok(8)) return launch_topk<T, 8, 1>(p, num_sms, st);
    if (E <= 512 && vec_ok(8)) return launch_topk<T, 8, 2>(p, num_sms, st);
    if (vec_ok(8)) return launch_topk<T, 8, 4>(p, num_sms, st);
  } else {
    if (E <= 256 && vec_ok(4)) return launch_topk<T, 4, 2>(p, num_sms, st);
    if (E <= 512 && vec_ok(4)) return launch_topk<T, 4, 4>(p, num_sms, st);
    if (vec_ok(4)) return launch_topk<T, 4, 8>(p, num_sms, st);
  }
  if (E <= 64) return launch_topk<T, 1, 2>(p, num_sms, st);
  if (E <= 256) return launch_topk<T, 1, 8>(p, num_sms, st);
  return launch_topk<T, 1, 32>(p, num_sms, st);
}

template <typename T, int L>
cudaError_t pick_grad(const RouteGradParams &p, int num_sms, cudaStream_t st) {
  constexpr int vec = 16 / (int)sizeof(T);
  const bool dense = p.softmax && !p.renormalize;
  const bool v = p.num_experts % vec == 0 && p.ld % vec == 0 && p.ld_grad % vec == 0 &&
                 reinterpret_cast<uintptr_t>(p.logits) % 16 == 0 &&
                 reinterpret_cast<uintptr_t>(p.grad_logits) % 16 == 0;
  const int64_t per_cta = (int64_t)kRouterWarps * (32 / L);
  const int64_t ctas = std::min<int64_t>((p.tokens + per_cta - 1) / per_cta, (int64_t)num_sms * 64);
  const dim3 grid((unsigned)ctas), block(kRouterWarps * 32);
  if (dense)
    return v ? launch_pdl(k_route_softmax_backward<T, L>, grid, block, 0, st, p)
             : launch_pdl(k_route_topk_backward<T, L, false, true>, grid, block, 0, st, p);
  return v ? launch_pdl(k_route_topk_backward<T, L, true, false>, grid, block, 0, st, p)
           : launch_pdl(k_route_topk_backward<T, L, false, false>, grid, block, 0, st, p);
}

}  // namespace

cudaError_t launch_route_topk(const RouteTopkParams &p, bool bf16, int num_sms, cudaStream_t st) {
  return bf16 ? pick_topk<__nv_bfloat16>(p, num_sms, st) : pick_topk<float>(p, num_sms, st);
}
cudaError_t launch_route_topk_backward(const RouteGradParams &p, bool bf16, int num_sms, cudaStream_t st) {
  if (p.top_k <= 8 && p.num_experts <= 256)
    return bf16 ? pick_grad<__nv_bfloat16, 8>(p, num_sms, st) : pick_grad<float, 8>(p, num_sms, st);
  return bf16 ? pick_grad<__nv_bfloat16, 32>(p, num_sms, st) : pick_grad<float, 32>(p, num_sms, st);
}

}  // namespace nvfp4
