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
// A warp per token.  A lane keeps its E/32 keys as order-preserving integers
// with the low bits replaced by the inverted expert index, so that a round of
// the selection is one warp-wide integer maximum (redux) that names the expert,
// and removing it is one compare per key.  When two neighbouring results (the
// first rejected key included) agree in every bit that is left of the key, the
// token's selection runs again on the whole keys.  bf16 logits without a bias
// lose no bits and never need that.
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

__device__ __forceinline__ float sigmoid(float x) { return 1.0f / (1.0f + expf(-x)); }

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

// ---------------------------------------------------------------- selection --
// Expert of a lane's value (c, i): c * 32 * VEC + lane * VEC + i.
template <typename T, int VEC, int NCH>
__global__ void __launch_bounds__(kRouterWarps * 32) k_route_topk(const RouteTopkParams p) {
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
        float key = x[v];
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
      w = id >= 0 ? sigmoid(xs) : 0.0f;
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

// ----------------------------------------------------------------- gradient --
// With d_j = scale * grad_w_j (0 for an id outside [0, E)) and the choice held fixed:
//   sigmoid:  ds_j = renormalize ? (d_j - sum_i d_i w_i) / S : d_j,  w_i = s_i / S,  S = sum_i s_i
//             dx_j = ds_j s_j (1 - s_j) on the chosen experts, 0 elsewhere
//   softmax, renormalized: the weights are the softmax over the chosen logits:
//             dx_j = w_j (d_j - sum_i d_i w_i) on the chosen experts, 0 elsewhere
//   softmax:  dx_e = p_e (d_e - sum_j d_j p_j) for every expert
// Each row of grad_logits is written whole: a warp lays its row out in shared
// memory (zeros, the chosen experts' values on top) and stores it in 16-byte
// vectors.  HBM-bound on that write (and, in the last form, the logits' read).
template <typename T, bool kVec, bool kDense>
__global__ void __launch_bounds__(kRouterWarps * 32) k_route_topk_backward(const RouteGradParams p) {
  griddep_launch_dependents();
  griddep_wait();   // inputs may come from the previous kernel in the stream
  extern __shared__ __align__(16) uint8_t sh_grad[];
  constexpr int VEC = kVec ? 16 / (int)sizeof(T) : 1;
  const int lane = threadIdx.x & 31;
  const int E = p.num_experts, k = p.top_k;
  // kDense: fp32 d_e of every expert; else the finished row in T
  using B = typename std::conditional<kDense, float, T>::type;
  B *buf = reinterpret_cast<B *>(sh_grad + (size_t)(threadIdx.x >> 5) * p.row_bytes);
  for (int e = lane; e < E; e += 32) store1(buf + e, 0.0f);
  __syncwarp();
  for (int64_t t = (int64_t)blockIdx.x * kRouterWarps + (threadIdx.x >> 5); t < p.tokens;
       t += (int64_t)gridDim.x * kRouterWarps) {
    const T *row = reinterpret_cast<const T *>(p.logits) + t * p.ld;
    T *out = reinterpret_cast<T *>(p.grad_logits) + t * p.ld_grad;
    int id = lane < k ? __ldg(p.expert_ids + t * k + lane) : -1;
    if (id >= E) id = -1;
    const float d = id >= 0 ? __ldg(p.grad_weights + t * k + lane) * p.scale : 0.0f;
    const float xs = id >= 0 ? load1(row + id) : -INFINITY;
    if constexpr (kDense) {
      float m = -INFINITY;
      for (int e = lane * VEC; e < E; e += 32 * VEC) {
        float x[VEC];
        load_vec<VEC>(row + e, x);
#pragma unroll
        for (int i = 0; i < VEC; ++i)
          if (x[i] > m) m = finite_top(x[i]);
      }
      m = warp_max(m);
      if (!(m > -INFINITY)) m = 0.0f;      // an empty row: every p is 0
      float s = 0.0f;
      for (int e = lane * VEC; e < E; e += 32 * VEC) {
        float x[VEC];
        load_vec<VEC>(row + e, x);
#pragma unroll
        for (int i = 0; i < VEC; ++i)
          if (x[i] > -INFINITY) s += expf(finite_top(x[i]) - m);
      }
      s = warp_sum(s);
      const float inv = s > 0.0f ? 1.0f / s : 0.0f;
      const float ps = xs > -INFINITY ? expf(finite_top(xs) - m) * inv : 0.0f;
      const float dot = warp_sum(d * ps);
      if (id >= 0) buf[id] = d;
      __syncwarp();
      for (int e = lane * VEC; e < E; e += 32 * VEC) {
        float x[VEC];
        load_vec<VEC>(row + e, x);
#pragma unroll
        for (int i = 0; i < VEC; ++i)
          x[i] = x[i] > -INFINITY ? expf(finite_top(x[i]) - m) * inv * (buf[e + i] - dot) : 0.0f;
        if constexpr (VEC == 8) {
          uint32_t o[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            o[i] = *reinterpret_cast<const uint32_t *>(&h);
          }
          *reinterpret_cast<uint4 *>(out + e) = make_uint4(o[0], o[1], o[2], o[3]);
        } else if constexpr (VEC == 4) {
          *reinterpret_cast<float4 *>(out + e) = make_float4(x[0], x[1], x[2], x[3]);
        } else {
          store1(out + e, x[0]);
        }
      }
      __syncwarp();
      if (id >= 0) buf[id] = 0.0f;
      __syncwarp();
    } else {
      float g = 0.0f;
      if (p.softmax) {                       // renormalized
        const float m = warp_max(finite_top(xs));
        const float e = xs > -INFINITY ? expf(finite_top(xs) - m) : 0.0f;
        const float s = warp_sum(e);
        const float w = s > 0.0f ? e / s : 0.0f;
        const float c = warp_sum(d * w);
        g = w * (d - c);
      } else {
        // s (1 - s) from exp(-|x|): 1 - s would cancel for large x
        const float a = expf(-fabsf(xs));
        const float slope = a / ((1.0f + a) * (1.0f + a));
        if (p.renormalize) {
          // slope / S <= 1 whatever the size of S: 1 / S alone may overflow
          const float s = id >= 0 ? sigmoid(xs) : 0.0f;
          const float S = warp_sum(s);
          const float c = warp_sum(S > 0.0f ? d * (s / S) : 0.0f);
          g = id >= 0 && S > 0.0f ? (d - c) * (slope / S) : 0.0f;
        } else {
          g = id >= 0 ? d * slope : 0.0f;
        }
      }
      if (id >= 0) store1(buf + id, g);
      __syncwarp();
      if constexpr (kVec) {
        for (int e = lane * VEC; e < E; e += 32 * VEC)
          *reinterpret_cast<uint4 *>(out + e) = *reinterpret_cast<const uint4 *>(buf + e);
      } else {
        for (int e = lane; e < E; e += 32) out[e] = buf[e];
      }
      __syncwarp();
      if (id >= 0) store1(buf + id, 0.0f);
      __syncwarp();
    }
  }
}

template <typename T, int VEC, int NCH>
cudaError_t launch_topk(const RouteTopkParams &p, int num_sms, cudaStream_t st) {
  const size_t smem = p.num_groups > 1 ? (size_t)kRouterWarps * p.num_experts * 4 : 0;   // <= 32 KB
  const int64_t ctas = std::min<int64_t>((p.tokens + kRouterWarps - 1) / kRouterWarps, (int64_t)num_sms * 8);
  return launch_pdl(k_route_topk<T, VEC, NCH>, dim3((unsigned)ctas), dim3(kRouterWarps * 32), smem, st, p);
}

// Values per lane by the number of experts; vector loads where the rows allow
// them (every row starts on the vector's size and E is a multiple of it).
template <typename T>
cudaError_t pick_topk(const RouteTopkParams &p, int num_sms, cudaStream_t st) {
  const int E = p.num_experts;
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

template <typename T>
cudaError_t pick_grad(const RouteGradParams &p0, int num_sms, cudaStream_t st) {
  RouteGradParams p = p0;
  constexpr int vec = 16 / (int)sizeof(T);
  const bool dense = p.softmax && !p.renormalize;
  const bool v = p.num_experts % vec == 0 && p.ld % vec == 0 && p.ld_grad % vec == 0 &&
                 reinterpret_cast<uintptr_t>(p.logits) % 16 == 0 &&
                 reinterpret_cast<uintptr_t>(p.grad_logits) % 16 == 0;
  p.row_bytes = (int)(((size_t)p.num_experts * (dense ? 4 : sizeof(T)) + 15) / 16 * 16);
  const size_t smem = (size_t)kRouterWarps * p.row_bytes;   // <= 32 KB
  const int64_t ctas = std::min<int64_t>((p.tokens + kRouterWarps - 1) / kRouterWarps, (int64_t)num_sms * 8);
  const dim3 grid((unsigned)ctas), block(kRouterWarps * 32);
  if (dense)
    return v ? launch_pdl(k_route_topk_backward<T, true, true>, grid, block, smem, st, p)
             : launch_pdl(k_route_topk_backward<T, false, true>, grid, block, smem, st, p);
  return v ? launch_pdl(k_route_topk_backward<T, true, false>, grid, block, smem, st, p)
           : launch_pdl(k_route_topk_backward<T, false, false>, grid, block, smem, st, p);
}

}  // namespace

cudaError_t launch_route_topk(const RouteTopkParams &p, bool bf16, int num_sms, cudaStream_t st) {
  return bf16 ? pick_topk<__nv_bfloat16>(p, num_sms, st) : pick_topk<float>(p, num_sms, st);
}
cudaError_t launch_route_topk_backward(const RouteGradParams &p, bool bf16, int num_sms, cudaStream_t st) {
  return bf16 ? pick_grad<__nv_bfloat16>(p, num_sms, st) : pick_grad<float>(p, num_sms, st);
}

}  // namespace nvfp4
