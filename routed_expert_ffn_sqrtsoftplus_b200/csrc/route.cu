// Routing from given logits, and its gradient.
//
//   s_e = softmax(z)_e | 1 / (1 + e^-z_e) | sqrt(log(1 + e^z_e))
//   selection by the keys s_e + b_e: the k largest, lower expert first on a tie, from
//   the topk_groups worthiest of G groups of E / G consecutive experts (worth: the
//   group's largest key, or the sum of its two largest; lower group first on a tie)
//   w_j = scale * s_j, or scale * s_j / sum of the selected s
// An expert whose logit is -inf is off. A slot that finds no expert gets -1 and
// weight 0. A row with NaN or +inf logits, or keys that are not finite, gets the
// placeholder experts 0..k-1 with NaN weights.
//
// One warp per row: the row is read once and kept in registers, lane l holding the
// consecutive experts l * EPL + i, so the lowest expert of a tie sits in the lowest
// lane. The selection works on order-preserving 32-bit keys (select_by_list).
//
// Exactness. Without a bias the three scores grow with the logit, so the logits
// themselves are the keys and the selection is exact. With a bias, or where a group is
// worth the sum of two scores, keys are 32-bit sums with a small error (kKeyTol). Where
// two neighbours of a row's selection are nearer than that, the experts that may belong
// to it, one per lane, are put in order by 64-bit keys (order_f64); where it is the groups
// that cannot be told apart, the experts that may count in their worth are (groups_f64). A row
// with more than 32 of either is selected from 64-bit keys as a whole (select_row_f64). So the
// result is always that of the 64-bit keys.
//
// Bound by instructions: 1080 a row of 256 FP32 logits with bias and groups (13.6 us for 8192 rows, of which HBM
// needs 1.3; 2.5 of 4 issue slots are taken while the SMs are busy, and a row in itself takes 3 us of latencies), 530
// a row of 128 BF16 logits without either (4.0 us for 4099 rows; HBM 0.2). A row takes a whole warp whatever E is: 16384 x
// 64 FP32 11.8 us (HBM 0.8); groups that lanes do not align with go through shared memory: 16384 x 200 BF16 in 8 groups
// 28.5 us (HBM 1.2).
#include <cuda_fp16.h>

#include "common.cuh"
#include "kernels.h"

namespace moe {

namespace {

constexpr int kRouteWarps = 4;  // rows per block
constexpr uint32_t kFull = 0xffffffffu;

// Two 32-bit keys may stand in the wrong order where they are no further apart than this, times key_base + |key|: the
// sum with the bias rounds with the key (half a unit of 2^-23 each), the scores' own errors do not shrink with what a
// bias leaves of them.
constexpr float kKeyTol = 2.384185791015625e-7f;  // 2^-22
// The error of two scores, in that unit. Sigmoid: __expf is off by 2 + 1.2 |x| units of 2^-23, of which u / (1 + u)^2
// (at most 0.6 units in all) reaches the score; the quotient and 1 + u add two at most. Softmax: the sum of up to
// 512 terms adds up to 21 roundings. sqrt(log(1 + e^z)) is not bounded: e^z is good to two units of 2^-23 of itself, its
// logarithm to one more, the sum with z to half of one; the root halves that and adds half a unit: at most 2.25 units of
// the score, which is sqrt(zmax + 0.7) at most.
__device__ __forceinline__ float key_base(int score, float zmax) {
  return score == kScoreSoftmax ? 16.0f : score == kScoreSigmoid ? 4.0f : 2.5f * sqrtf(fmaxf(zmax, 0.0f) + 0.7f);
}

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<float>(float v) {
  return v;
}
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) {
  return __bfloat162float(v);
}
template <>
__device__ __forceinline__ float to_f32<__half>(__half v) {
  return __half2float(v);
}
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) {
  return v;
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) {
  return __float2half_rn(v);
}

// EPL consecutive elements from p (vec: p is aligned to the vector width below and all EPL exist).
template <typename T, int EPL>
__device__ __forceinline__ void load_run(const T* p, int n, bool vec, float (&z)[EPL]) {
  constexpr int kBytes = EPL * static_cast<int>(sizeof(T));
  if (vec && n >= EPL) {
    if constexpr (kBytes % 16 == 0) {
#pragma unroll
      for (int q = 0; q < kBytes / 16; ++q) {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(p) + q);
        const T* t = reinterpret_cast<const T*>(&v);
#pragma unroll
        for (int i = 0; i < 16 / static_cast<int>(sizeof(T)); ++i) z[q * (16 / sizeof(T)) + i] = to_f32<T>(t[i]);
      }
    } else {
#pragma unroll
      for (int q = 0; q < kBytes / 8; ++q) {
        const uint2 v = __ldg(reinterpret_cast<const uint2*>(p) + q);
        const T* t = reinterpret_cast<const T*>(&v);
#pragma unroll
        for (int i = 0; i < 8 / static_cast<int>(sizeof(T)); ++i) z[q * (8 / sizeof(T)) + i] = to_f32<T>(t[i]);
      }
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < EPL; ++i) z[i] = i < n ? to_f32<T>(p[i]) : -INFINITY;
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
  return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}

// Order-preserving map of floats to unsigned: 0 is below every float (an expert that is off).
__device__ __forceinline__ uint32_t key_of(float v) {
  const uint32_t b = __float_as_uint(v + 0.0f);  // -0 and +0 are equal
  return b ^ ((b & 0x80000000u) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t k) {
  return __uint_as_float(k ^ ((k & 0x80000000u) ? 0x80000000u : 0xffffffffu));
}

__device__ __forceinline__ float sigmoid_f32(float z) {
  const float u = expf(-fabsf(z));
  return __fdiv_rn(z >= 0.0f ? 1.0f : u, 1.0f + u);
}
__device__ __forceinline__ float score_f32(float z, int score, float m, float inv_sum) {
  if (score == kScoreSoftmax) return expf(z - m) * inv_sum;
  if (score == kScoreSigmoid) return sigmoid_f32(z);
  // far down log(1 + e^z) is e^z (to e^z / 2 of itself), whose root is an ordinary number where e^z is none
  if (z < -20.0f) return expf(0.5f * z);
  return sqrtf(fmaxf(z, 0.0f) + log1pf(expf(-fabsf(z))));
}
// The same for keys, whose error is an absolute one.
__device__ __forceinline__ float key_score(float z, int score, float m, float inv_sum) {
  if (score == kScoreSigmoid) {
    const float u = __expf(-fabsf(z));
    return __fdividef(z >= 0.0f ? 1.0f : u, 1.0f + u);
  }
  if (score == kScoreSoftmax) return expf(z - m) * inv_sum;
  return sqrtf(fmaxf(z, 0.0f) + log1pf(expf(-fabsf(z))));
}
__device__ __forceinline__ double score_f64(double z, int score, double m, double sum) {
  if (score == kScoreSoftmax) return exp(z - m) / sum;
  if (score == kScoreSigmoid) {
    const double u = exp(-fabs(z));
    return (z >= 0.0 ? 1.0 : u) / (1.0 + u);
  }
  return sqrt(fmax(z, 0.0) + log1p(exp(-fabs(z))));
}

// Scores of selected experts up to one factor that all of a row's share (it falls out
// of renormalised weights): with m = the largest selected logit, s_j divided by e^m
// (softmax), e^min(m, 0) (sigmoid) or e^(min(m, 0) / 2) (sqrtsoftplus), so that no row,
// however low its logits, divides zero by zero.
__device__ __forceinline__ float shared_score(float z, int score, float m) {
  if (score == kScoreSoftmax) return expf(z - m);
  const float low = fminf(m, 0.0f);
  if (score == kScoreSigmoid) return __fdiv_rn(expf(fminf(z, 0.0f) - low), 1.0f + expf(-fabsf(z)));
  if (z > 0.0f) return sqrtf(z + log1pf(expf(-z)));
  const float u = expf(z);
  const float r = u > 0.0f ? __fdiv_rn(log1pf(u), u) : 1.0f;  // log(1 + u) / u
  return expf(0.5f * (z - low)) * sqrtf(r);
}

struct SelectArgs {
  int E, G, kept, k, score, sum2;
  int Eg;          // experts of a group
  int lane_shift;  // a group is 2^lane_shift whole lanes, or -1
  int scan_shift;  // else 2^scan_shift lanes scan it (G groups: at most 32 lanes)
};

// Maximum and sum of a softmax row in 64 bits.
template <typename T>
__device__ __forceinline__ void softmax_f64(const T* row, int E, int lane, double& m, double& sum) {
  m = -INFINITY;
  sum = 0.0;
  for (int e = lane; e < E; e += 32) m = fmax(m, static_cast<double>(to_f32<T>(row[e])));
  for (int o = 16; o > 0; o >>= 1) m = fmax(m, __shfl_xor_sync(kFull, m, o));
  for (int e = lane; e < E; e += 32) sum += exp(static_cast<double>(to_f32<T>(row[e])) - m);
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
}

// The experts of lanes 0 .. n - 1 in the order of their 64-bit keys: lane r gets the r-th, or -1.
template <typename T>
__device__ __noinline__ int order_f64(const T* row, const float* bias, int E, int score, int cand, int n, int lane) {
  double m = 0.0, sum = 1.0;
  if (score == kScoreSoftmax) softmax_f64<T>(row, E, lane, m, sum);
  const bool has = lane < n;
  const double key = has ? score_f64(static_cast<double>(to_f32<T>(row[cand])), score, m, sum) +
                               (bias ? static_cast<double>(bias[cand]) : 0.0)
                         : -INFINITY;
  int rank = 0;
#pragma unroll 4
  for (int j = 0; j < n; ++j) {
    const double o = __shfl_sync(kFull, key, j);
    const int oc = __shfl_sync(kFull, cand, j);
    rank += o > key || (o == key && oc < cand);
  }
  int mine = -1;
#pragma unroll 4
  for (int j = 0; j < n; ++j) {
    const int oc = __shfl_sync(kFull, cand, j), orank = __shfl_sync(kFull, rank, j);
    if (orank == lane) mine = oc;
  }
  return mine;
}

// The kept groups (a mask) by the 64-bit keys of the experts of lanes 0 .. n - 1, which hold every group's
// largest two.
template <typename T>
__device__ __noinline__ uint32_t groups_f64(const T* row, const float* bias, SelectArgs a, int cand, int n, int lane) {
  double m = 0.0, sum = 1.0;
  if (a.score == kScoreSoftmax) softmax_f64<T>(row, a.E, lane, m, sum);
  const bool has = lane < n;
  const double key = has ? score_f64(static_cast<double>(to_f32<T>(row[cand])), a.score, m, sum) +
                               (bias ? static_cast<double>(bias[cand]) : 0.0)
                         : -INFINITY;
  const int group = has ? cand / (a.E / a.G) : -1;
  double w1 = -INFINITY, w2 = -INFINITY;
#pragma unroll 4
  for (int j = 0; j < n; ++j) {
    const double o = __shfl_sync(kFull, key, j);
    if (__shfl_sync(kFull, group, j) == lane) {
      w2 = fmax(w2, fmin(w1, o));
      w1 = fmax(w1, o);
    }
  }
  const double worth = a.sum2 && w2 != -INFINITY ? w1 + w2 : w1;
  int rank = 0;
  for (int g = 0; g < a.G; ++g) {
    const double o = __shfl_sync(kFull, worth, g);
    rank += o > worth || (o == worth && g < lane);
  }
  return __ballot_sync(kFull, lane < a.G && rank < a.kept);
}

// The j-th (from 0) of a warp's flags gathered so far: which of its elements a lane takes.
struct Gather {
  int cand = -1, total = 0;
  __device__ __forceinline__ void add(bool in, int lane, int epl, int i) {
    const uint32_t who = __ballot_sync(kFull, in);
    const int at = lane - total;
    if (at >= 0 && at < __popc(who)) cand = static_cast<int>(__fns(who, 0, at + 1)) * epl + i;
    total += __popc(who);
  }
};

// The selection from 64-bit keys held in `buf` (E doubles): lane r < k gets slot r's expert or -1.
template <typename T>
__device__ __noinline__ int select_row_f64(const T* row, const float* bias, SelectArgs a, double* buf, int lane) {
  double m = 0.0, sum = 1.0;
  if (a.score == kScoreSoftmax) softmax_f64<T>(row, a.E, lane, m, sum);
  for (int e = lane; e < a.E; e += 32) {
    const double z = to_f32<T>(row[e]);
    buf[e] = z == -INFINITY ? -INFINITY
                            : score_f64(z, a.score, m, sum) + (bias ? static_cast<double>(bias[e]) : 0.0);
  }
  __syncwarp();
  const int Eg = a.E / a.G;
  uint32_t keep = kFull;
  if (a.kept < a.G) {
    double w1 = -INFINITY, w2 = -INFINITY;
    if (lane < a.G)
      for (int j = 0; j < Eg; ++j) {
        const double v = buf[lane * Eg + j];
        if (v > w1) {
          w2 = w1;
          w1 = v;
        } else if (v > w2) {
          w2 = v;
        }
      }
    const double worth = a.sum2 && w2 != -INFINITY ? w1 + w2 : w1;
    int rank = 0;
    for (int g = 0; g < a.G; ++g) {
      const double o = __shfl_sync(kFull, worth, g);
      rank += o > worth || (o == worth && g < lane);
    }
    keep = __ballot_sync(kFull, lane < a.G && rank < a.kept);
    if (bias == nullptr) {  // the logits are the keys, only the groups' worth is a sum of scores
      for (int e = lane; e < a.E; e += 32) buf[e] = to_f32<T>(row[e]);
      __syncwarp();
    }
  }
  int mine = -1;
  for (int r = 0; r < a.k; ++r) {
    double bv = -INFINITY;
    int bi = 0x7fffffff;
    for (int e = lane; e < a.E; e += 32)
      if (((keep >> (e / Eg)) & 1u) && buf[e] > bv) {
        bv = buf[e];
        bi = e;
      }
    for (int o = 16; o > 0; o >>= 1) {
      const double ov = __shfl_xor_sync(kFull, bv, o);
      const int oi = __shfl_xor_sync(kFull, bi, o);
      if (ov > bv || (ov == bv && oi < bi)) {
        bv = ov;
        bi = oi;
      }
    }
    if (bi == 0x7fffffff) break;  // nothing is left: the slots from r on stay empty
    if (lane == r) mine = bi;
    if (bi % 32 == lane) buf[bi] = -INFINITY;
    __syncwarp();
  }
  return mine;
}

// The k largest of the warp's keys (0: none) in order, lower expert first on a tie: lane r gets the r-th
// expert and key, `left` the largest key left (0 if there is none); how many there are is returned.
//
// In rounds: a warp maximum (redux.sync) finds the next, and its lane looks for its next one.
template <int EPL>
__device__ __forceinline__ int select_by_rounds(uint32_t (&key)[EPL], int e0, int k, int lane, int& mine,
                                                uint32_t& mkey, uint32_t& left) {
  uint32_t bk = 0u;
  int bi = 0, n = 0;
#pragma unroll
  for (int i = 0; i < EPL; ++i)
    if (key[i] > bk) {
      bk = key[i];
      bi = i;
    }
#pragma unroll 1
  for (;; ++n) {
    const uint32_t m = __reduce_max_sync(kFull, bk);
    left = m;
    if (n == k || m == 0u) break;
    if (lane == n) mkey = m;
    const int win = __ffs(__ballot_sync(kFull, bk == m)) - 1;
    const int e = __shfl_sync(kFull, e0 + bi, win);
    if (lane == n) mine = e;
    if (lane == win) {
      const int was = bi;
      bk = 0u;
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        if (i == was) key[i] = 0u;
        if (key[i] > bk) {
          bk = key[i];
          bi = i;
        }
      }
    }
  }
  return n;
}

// By a list: the k-th largest of the lanes' maxima (with 12 keys a lane or more, of their halves' maxima)
// bounds the k-th largest key from below, and few keys reach that bound. They go to a list of at most 32 (key, expert), one a lane, and each counts those ahead of
// it. -1 where there are more; `base` (key_base, or 0 for keys that are exact) lowers the bound, so that the list also holds what
// floats cannot tell from the last slot. Some 200 instructions where rounds take 60 each.
//
// Halves where they are long: of 512 experts in 8 groups, 4 of them kept, 16 lanes are live, and a list for 16
// slots by their maxima is the 256 keys of them all (16384 rows in rounds: 72.6 us, by halves 46.9; by halves
// without groups, 12 slots, 26.5 against 25.6). Above 16 slots the bound lets too many through either way.
constexpr int kListK = 16;
template <int EPL>
__device__ __forceinline__ int select_by_list(const uint32_t (&key)[EPL], int e0, int k, float base, uint2* list,
                                              int lane, int& mine, uint32_t& mkey, uint32_t& left) {
  constexpr int kParts = EPL >= 12 ? 2 : 1, kLen = EPL / kParts;
  uint32_t bk[kParts];
  int live = 0;
#pragma unroll
  for (int h = 0; h < kParts; ++h) {
    bk[h] = 0u;
#pragma unroll
    for (int i = 0; i < kLen; ++i) bk[h] = max(bk[h], key[h * kLen + i]);
    live += __popc(__ballot_sync(kFull, bk[h] != 0u));
  }
  // the k-th maximum of few more than k parts (the others' groups are out) is a low one: the list would
  // overflow (of 4 k / 3 parts with 16 keys each some 21 reach it, of k parts all)
  if (4 * k > 3 * live && live * kLen > 32) return -1;
  uint32_t bound = 0u;
  int reached = 0;
  for (int r = 0; r < k && reached < k; ++r) {  // equal maxima go together
    uint32_t most = bk[0];
#pragma unroll
    for (int h = 1; h < kParts; ++h) most = max(most, bk[h]);
    bound = __reduce_max_sync(kFull, most);
#pragma unroll
    for (int h = 0; h < kParts; ++h) {
      const bool top = bk[h] == bound;
      reached += __popc(__ballot_sync(kFull, top));
      if (top) bk[h] = 0u;
    }
  }
  // fewer than k parts with live experts: everything live
  if (reached < k || bound == 0u) bound = 1u;
  if (base > 0.f && bound > 1u) {
    const float f = value_of(bound);
    bound = max(1u, key_of(f - kKeyTol * (base + fabsf(f))));
  }
  int n = 0;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const bool in = key[i] >= bound;
    const uint32_t who = __ballot_sync(kFull, in);
    const int at = n + __popc(who & ((1u << lane) - 1u));
    if (in && at < 32) list[at] = make_uint2(key[i], static_cast<uint32_t>(e0 + i));
    n += __popc(who);
  }
  if (n > 32) return -1;
  __syncwarp();
  const uint2 my = lane < n ? list[lane] : make_uint2(0u, 0x7FFFFFFFu);
  int rank = 0;
#pragma unroll 4
  for (int j = 0; j < n; ++j) {
    const uint2 o = list[j];
    rank += o.x > my.x || (o.x == my.x && o.y < my.y);
  }
  __syncwarp();
  if (lane < n) list[rank] = my;
  __syncwarp();
  if (lane < min(n, k)) {
    const uint2 o = list[lane];
    mkey = o.x;
    mine = static_cast<int>(o.y);
  }
  left = n > k ? list[k].x : 0u;
  return min(n, k);
}

// The second bound keeps the widest rows at the registers of 5 and 6 blocks an SM (16384 x 512, 12 BF16 slots 26.4 us;
// 31.7 with the 108 registers that the compiler takes without it).
template <typename T, int EPL>
__global__ void __launch_bounds__(kRouteWarps * 32, EPL < 16 ? 1 : sizeof(T) == 4 ? 5 : 6)
    route_kernel(const T* __restrict__ logits, int64_t row_stride, const float* __restrict__ bias, int rows,
                 SelectArgs a, int renorm, float scale, int vec, int vec_bias, int32_t* __restrict__ idx_out,
                 float* __restrict__ w_out) {
  extern __shared__ double key_buf[];  // E doubles per warp, where keys are sums
  __shared__ uint2 list_buf[kRouteWarps][32];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int t = blockIdx.x * kRouteWarps + warp;
  if (t >= rows) return;
  const T* row = logits + static_cast<size_t>(t) * row_stride;
  const int e0 = lane * EPL;
  float z[EPL];
  load_run<T, EPL>(row + e0, min(EPL, a.E - e0), vec != 0, z);

  bool bad = false;
  float zmax = -INFINITY;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    bad |= !(z[i] < INFINITY);
    zmax = fmaxf(zmax, z[i]);
  }
  const bool grouped = a.kept < a.G;
  const bool need_scores = bias != nullptr || (grouped && a.sum2);
  float inv_sum = 1.0f;
  float base = 0.0f;
  if (need_scores) base = key_base(a.score, value_of(__reduce_max_sync(kFull, key_of(zmax))));
  if (a.score == kScoreSoftmax) {
    zmax = warp_max(zmax);
    if (need_scores || !renorm) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < EPL; ++i) s += z[i] == -INFINITY ? 0.f : expf(z[i] - zmax);
      inv_sum = __fdiv_rn(1.0f, warp_sum(s));
    }
  }
  // keys: the scores plus bias where there is one (v), else the logits
  uint32_t key[EPL];
  float v[EPL];
  if (bias != nullptr) load_run<float, EPL>(bias + e0, min(EPL, a.E - e0), vec_bias != 0, v);
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const bool live = z[i] != -INFINITY;
    const float b = bias != nullptr ? v[i] : 0.f;
    v[i] = z[i];
    if (need_scores && live) v[i] = key_score(z[i], a.score, zmax, inv_sum);
    if (bias != nullptr && live) {
      v[i] += b;
      bad |= !(fabsf(v[i]) < INFINITY);
    }
    key[i] = live ? key_of(bias != nullptr ? v[i] : z[i]) : 0u;
  }
  if (__any_sync(kFull, bad)) {
    if (lane < a.k) {
      idx_out[static_cast<size_t>(t) * a.k + lane] = lane;
      w_out[static_cast<size_t>(t) * a.k + lane] = __int_as_float(0x7fc00000);
    }
    return;
  }

  bool unsure = false;  // two neighbours of a choice nearer than 32-bit keys tell
  if (grouped) {
    const int Eg = a.Eg;
    // a group is a power of two of whole lanes: 2^lane_shift of them
    const bool whole = a.lane_shift >= 0;
    float w1 = -INFINITY, w2 = -INFINITY;
    // the two largest of 2^shift lanes each, then lane g takes group g's
    auto merge = [&](int shift) {
      for (int o = 1; o < 1 << shift; o <<= 1) {
        const float o1 = __shfl_xor_sync(kFull, w1, o), o2 = __shfl_xor_sync(kFull, w2, o);
        w2 = fmaxf(fmaxf(w2, o2), fminf(w1, o1));
        w1 = fmaxf(w1, o1);
      }
      const int src = min(lane, a.G - 1) << shift;
      w1 = __shfl_sync(kFull, w1, src);
      w2 = __shfl_sync(kFull, w2, src);
    };
    if (whole) {
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        w2 = fmaxf(w2, fminf(w1, v[i]));
        w1 = fmaxf(w1, v[i]);
      }
      merge(a.lane_shift);
    } else {
      float* fb = reinterpret_cast<float*>(key_buf + static_cast<size_t>(warp) * a.E);  // this warp's alone
      // lanes EPL apart, each on a bank of its own (16384 x 480, 8 groups: 50.2 us, 56.9 without)
      auto pad = [](int e) { return e + (e >> 4); };
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        if (e0 + i < a.E) fb[pad(e0 + i)] = v[i];
      __syncwarp();
      // 2^scan_shift lanes scan a group
      const int g = lane >> a.scan_shift, step = 1 << a.scan_shift;
      if (g < a.G)
        for (int j = lane & (step - 1); j < Eg; j += step) {
          const float x = fb[pad(g * Eg + j)];
          w2 = fmaxf(w2, fminf(w1, x));
          w1 = fmaxf(w1, x);
        }
      merge(a.scan_shift);
      __syncwarp();
    }
    // half of the sum of two keys (the sum of two of the type's lowest values would be -infinity), off by
    // no more than err
    const bool two = a.sum2 && w2 != -INFINITY;
    float worth = a.sum2 ? 0.5f * w1 + 0.5f * (two ? w2 : 0.f) : w1;
    const float err = 0.5f * kKeyTol * (base + (two ? 0.5f * fabsf(w1) + 0.5f * fabsf(w2) : fabsf(w1)));
    if (lane >= a.G) worth = -INFINITY;
    int rank = 0;
#pragma unroll 4
    for (int g = 0; g < a.G; ++g) {
      const float o = __shfl_sync(kFull, worth, g);
      rank += o > worth || (o == worth && g < lane);
    }
    const bool in = lane < a.G && rank < a.kept;
    uint32_t keep = __ballot_sync(kFull, in);
    if (need_scores) {
      // the least that a kept group may be worth, and the most that another may
      const uint32_t least = __reduce_min_sync(kFull, in ? key_of(worth - err) : kFull);
      const uint32_t most = __reduce_max_sync(kFull, in || worth == -INFINITY ? 0u : key_of(worth + err));
      if (least <= most) {
        // of each group, what reaches its second (or its first) key
        const float low = a.sum2 && w2 != -INFINITY ? w2 : w1;
        const float from = lane < a.G ? low - kKeyTol * (base + fabsf(low)) : INFINITY;
        Gather cands;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
          const float f = __shfl_sync(kFull, from, min(e0 + i, a.E - 1) / Eg);
          cands.add(v[i] != -INFINITY && v[i] >= f, lane, EPL, i);
        }
        if (cands.total <= 32)
          keep = groups_f64<T>(row, bias, a, cands.cand, cands.total, lane);
        else
          unsure = true;
      }
    }
    if (whole) {
      const bool out = !((keep >> (lane >> a.lane_shift)) & 1u);
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        if (out) {
          key[i] = 0u;
          v[i] = -INFINITY;
        }
    } else {
      int g = e0 / Eg, left = Eg - e0 % Eg;
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        if (e0 + i < a.E && !((keep >> g) & 1u)) {
          key[i] = 0u;
          v[i] = -INFINITY;
        }
        if (--left == 0) {
          ++g;
          left = Eg;
        }
      }
    }
  }

  int mine = -1, n = 0;  // slot `lane`'s expert; slots filled
  uint32_t mkey = 0u, left = 0u;  // its key, and the best one left
  if (a.k <= kListK)
    n = select_by_list<EPL>(key, e0, a.k, bias != nullptr ? base : 0.f, list_buf[warp], lane, mine, mkey, left);
  if (a.k > kListK || n < 0) n = select_by_rounds<EPL>(key, e0, a.k, lane, mine, mkey, left);
  if (bias != nullptr) {
    // neighbours that 32-bit keys do not tell apart: order what reaches down to the last slot's key again
    uint32_t next = __shfl_down_sync(kFull, mkey, 1);
    if (lane == n - 1) next = left;
    const float mine_f = value_of(mkey);
    const bool close = lane < n && next != 0u && mine_f - value_of(next) <= kKeyTol * (base + fabsf(mine_f));
    if (!unsure && __any_sync(kFull, close)) {
      const float last = __shfl_sync(kFull, mine_f, n - 1);
      const float least = last - kKeyTol * (base + fabsf(last));
      Gather cands;
#pragma unroll
      for (int i = 0; i < EPL; ++i)  // with a bias v holds the keys, -infinity where the expert is out
        cands.add(v[i] != -INFINITY && v[i] >= least, lane, EPL, i);
      if (cands.total <= 32)
        mine = order_f64<T>(row, bias, a.E, a.score, cands.cand, cands.total, lane);
      else
        unsure = true;
      if (lane >= a.k) mine = -1;
    }
  }
  if (unsure) mine = select_row_f64<T>(row, bias, a, key_buf + static_cast<size_t>(warp) * a.E, lane);

  const bool has = mine >= 0;
  const float zs = has ? to_f32<T>(row[mine]) : -INFINITY;
  float w = 0.f;
  if (renorm) {
    const float m = warp_max(zs);
    const float s = has ? shared_score(zs, a.score, m) : 0.f;
    const float sum = warp_sum(s);
    if (has) w = scale * __fdiv_rn(s, sum);
  } else if (has) {
    w = scale * score_f32(zs, a.score, zmax, inv_sum);
  }
  if (lane < a.k) {
    idx_out[static_cast<size_t>(t) * a.k + lane] = mine;
    w_out[static_cast<size_t>(t) * a.k + lane] = w;
  }
}

// Gradient of the logits from the weights' gradients g, the selection held fixed. With
// p_j = s_j / S the renormalised scores and gbar = sum_j g_j p_j:
//   renormalised: softmax       dz_j = scale p_j (g_j - gbar)
//                 sigmoid       dz_j = scale p_j (g_j - gbar) (1 - s_j)
//                 sqrtsoftplus  dz_j = scale p_j (g_j - gbar) sigmoid(z_j) / (2 softplus(z_j))
//   otherwise:    sigmoid, sqrtsoftplus: s_j in the place of p_j and gbar = 0
//                 softmax       dz_e = s_e (scale g_e [e selected] - scale sum_j g_j s_j), every e
// One warp per row; lane r holds slot r (an expert named twice adds up). The row is written 16 bytes a
// lane without the slots' own terms (zeros, or in the dense form -s_e scale sum_j g_j s_j from a row held
// in registers), and the slots' elements go over it: one warp, so in this order. Bound by HBM's writes: 16384 x
// 512 FP32, 16 slots, 8.9 us (HBM 5.6), dense 13.5 (10.6; 39 with the row read and exponentiated twice).
template <typename T, bool kDense>
__global__ void __launch_bounds__(kRouteWarps * 32)
    route_grad_kernel(const float* __restrict__ grad_w, const T* __restrict__ logits, int64_t row_stride,
                      const int32_t* __restrict__ idx, int rows, int E, int k, int score, int renorm, float scale,
                      int vec_in, int vec_out, T* __restrict__ out) {
  constexpr int V = 16 / static_cast<int>(sizeof(T));
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int t = blockIdx.x * kRouteWarps + warp;
  if (t >= rows) return;
  const T* row = logits + static_cast<size_t>(t) * row_stride;
  int e = lane < k ? __ldg(idx + static_cast<size_t>(t) * k + lane) : -1;
  if (e >= E) e = -1;  // not an expert: no gradient, and no read outside the row
  const bool has = e >= 0;
  const float g = has ? __ldg(grad_w + static_cast<size_t>(t) * k + lane) : 0.f;
  const float zs = has ? to_f32<T>(row[e]) : -INFINITY;
  float d = 0.f;  // the slot's gradient
  T* orow = out + static_cast<size_t>(t) * E;
  // an expert named twice: its first slot takes the sum
  const uint32_t same = __match_any_sync(kFull, e);
  const bool lead = has && __ffs(same) - 1 == lane;
  const bool twice = __any_sync(kFull, has && (same & (same - 1)) != 0u);
  auto join = [&]() {
    float sum = 0.f;
    for (int r = 0; r < k; ++r) {
      const float dr = __shfl_sync(kFull, d, r);
      if ((same >> r) & 1u) sum += dr;
    }
    d = sum;
  };
  if constexpr (kDense) {
    // the row in registers: its exponentials are taken once
    constexpr int kChunks = 512 / (32 * V);
    float z[kChunks][V];
    float zmax = -INFINITY, s = 0.f;
#pragma unroll
    for (int u = 0; u < kChunks; ++u) {
      const int c = (u * 32 + lane) * V;
      load_run<T, V>(row + c, min(V, E - c), vec_in != 0, z[u]);
#pragma unroll
      for (int i = 0; i < V; ++i) zmax = fmaxf(zmax, z[u][i]);
    }
    zmax = warp_max(zmax);
#pragma unroll
    for (int u = 0; u < kChunks; ++u)
      if (u * 32 * V < E) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          z[u][i] = z[u][i] == -INFINITY ? 0.f : expf(z[u][i] - zmax);  // an expert that is off, and a row of them: 0
          s += z[u][i];
        }
      }
    s = warp_sum(s);
    const float inv_sum = s > 0.f || s != s ? __fdiv_rn(1.0f, s) : 0.f;
    const float sj = has && zs != -INFINITY ? expf(zs - zmax) * inv_sum : 0.f;
    d = scale * g;
    const float back = warp_sum(d * sj);
#pragma unroll
    for (int u = 0; u < kChunks; ++u) {
      const int c = (u * 32 + lane) * V;
      if (c >= E) break;
#pragma unroll
      for (int i = 0; i < V; ++i) z[u][i] = -(z[u][i] * inv_sum) * back;
      if (vec_out && c + V <= E) {
        uint4 o;
        T* ot = reinterpret_cast<T*>(&o);
#pragma unroll
        for (int i = 0; i < V; ++i) ot[i] = from_f32<T>(z[u][i]);
        *reinterpret_cast<uint4*>(orow + c) = o;
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (c + i < E) orow[c + i] = from_f32<T>(z[u][i]);
      }
    }
    if (twice) join();
    d = sj * (d - back);
  } else {
    float p, gbar = 0.f;
    if (renorm) {
      const float m = warp_max(zs);
      p = has && zs != -INFINITY ? shared_score(zs, score, m) : 0.f;
      const float sum = warp_sum(p);
      p = sum > 0.f || sum != sum ? __fdiv_rn(p, sum) : 0.f;
      gbar = warp_sum(g * p);
    } else {
      p = has ? score_f32(zs, score, 0.f, 1.f) : 0.f;
    }
    float slope = 1.0f;
    if (score == kScoreSigmoid) {
      slope = sigmoid_f32(-zs);
    } else if (score == kScoreSqrtSoftplus) {
      const float u = expf(-fabsf(zs));
      // sigmoid / softplus; for z <= 0 both over e^z, so that it tends to 1
      slope = zs > 0.f ? __fdiv_rn(1.0f, (1.0f + u) * (zs + log1pf(u)))
                       : __fdiv_rn(1.0f, (1.0f + u) * (u > 0.f ? __fdiv_rn(log1pf(u), u) : 1.0f));
      slope *= 0.5f;
    }
    d = has ? scale * p * (g - gbar) * slope : 0.f;
    if (twice) join();
    for (int c = lane * V; c < E; c += 32 * V) {
      if (vec_out && c + V <= E) {
        *reinterpret_cast<uint4*>(orow + c) = make_uint4(0u, 0u, 0u, 0u);
      } else {
        for (int i = 0; i < V && c + i < E; ++i) orow[c + i] = from_f32<T>(0.f);
      }
    }
  }
  __syncwarp();
  if (lead) orow[e] = from_f32<T>(d);
}

template <typename T, int EPL>
cudaError_t launch_route_epl(const RouteArgs& r, cudaStream_t s) {
  constexpr int kBytes = EPL * static_cast<int>(sizeof(T));
  const uintptr_t vb = kBytes % 16 == 0 ? 16 : 8;
  const bool vec = reinterpret_cast<uintptr_t>(r.logits) % vb == 0 && (r.row_stride * sizeof(T)) % vb == 0;
  const bool grouped = r.topk_groups < r.n_groups;
  // 64-bit keys of the rows that need them, and the groups' keys where lanes do not align with groups
  const bool need = grouped || r.bias != nullptr;
  const size_t smem = need ? static_cast<size_t>(kRouteWarps) * r.E * sizeof(double) : 0;
  const int Eg = r.E / r.n_groups, lanes = Eg / EPL;
  int shift = -1;
  if (Eg % EPL == 0 && (lanes & (lanes - 1)) == 0)
    for (shift = 0; 1 << shift < lanes;) ++shift;
  int scan = 0;
  while (r.n_groups << (scan + 1) <= 32) ++scan;
  const SelectArgs a{r.E, r.n_groups, r.topk_groups, r.k, r.score, r.group_sum2, Eg, shift, scan};
  route_kernel<T, EPL><<<(r.T - 1) / kRouteWarps + 1, kRouteWarps * 32, smem, s>>>(
      static_cast<const T*>(r.logits), r.row_stride, r.bias, r.T, a, r.renorm, r.scale, vec ? 1 : 0,
      reinterpret_cast<uintptr_t>(r.bias) % 16 == 0 ? 1 : 0, r.idx, r.w);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_route_t(const RouteArgs& r, cudaStream_t s) {
  if (r.E <= 128) return launch_route_epl<T, 4>(r, s);
  if (r.E <= 256) return launch_route_epl<T, 8>(r, s);
  if (r.E <= 384) return launch_route_epl<T, 12>(r, s);
  return launch_route_epl<T, 16>(r, s);
}

template <typename T>
cudaError_t launch_route_grad_t(const RouteGradArgs& r, cudaStream_t s) {
  const bool vi = reinterpret_cast<uintptr_t>(r.logits) % 16 == 0 && (r.row_stride * sizeof(T)) % 16 == 0;
  const bool vo = reinterpret_cast<uintptr_t>(r.out) % 16 == 0 && (r.E * sizeof(T)) % 16 == 0;
  const bool dense = r.score == kScoreSoftmax && !r.renorm;
  auto* kernel = dense ? route_grad_kernel<T, true> : route_grad_kernel<T, false>;
  kernel<<<(r.T - 1) / kRouteWarps + 1, kRouteWarps * 32, 0, s>>>(
      r.grad_w, static_cast<const T*>(r.logits), r.row_stride, r.idx, r.T, r.E, r.k, r.score, r.renorm, r.scale,
      vi ? 1 : 0, vo ? 1 : 0, static_cast<T*>(r.out));
  return cudaGetLastError();
}

// A caller's routing into the layer's own buffers. -1 is an empty slot; any other index
// outside [0, E) gets the slot's placeholder expert with a NaN weight and is reported.
__global__ void __launch_bounds__(256)
    take_routing_kernel(const int32_t* __restrict__ idx_in, const float* __restrict__ w_in, int n, int k, int E,
                        int32_t* __restrict__ idx, float* __restrict__ w, int* status) {
  const int i = blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= n) return;
  int e = idx_in[i];
  float wi = w_in[i];
  if (e < -1 || e >= E) {
    report_status(status, kStatusDevice);
    e = i % k;
    wi = __int_as_float(0x7fc00000);
  }
  idx[i] = e;
  w[i] = wi;
}

}  // namespace

cudaError_t launch_route(const RouteArgs& r, cudaStream_t s) {
  if (r.T == 0) return cudaSuccess;
  if (r.E > 512 || r.k > 32 || r.n_groups > 32) return cudaErrorInvalidValue;
  if (r.dtype == kValFp32) return launch_route_t<float>(r, s);
  if (r.dtype == kValBf16) return launch_route_t<__nv_bfloat16>(r, s);
  return launch_route_t<__half>(r, s);
}

cudaError_t launch_route_grad(const RouteGradArgs& r, cudaStream_t s) {
  if (r.T == 0) return cudaSuccess;
  if (r.k > 32 || r.E > 512) return cudaErrorInvalidValue;
  if (r.dtype == kValFp32) return launch_route_grad_t<float>(r, s);
  if (r.dtype == kValBf16) return launch_route_grad_t<__nv_bfloat16>(r, s);
  return launch_route_grad_t<__half>(r, s);
}

cudaError_t launch_take_routing(const int32_t* idx_in, const float* w_in, int T, int k, int E, int32_t* idx, float* w,
                                int* status, cudaStream_t s) {
  const int n = T * k;
  take_routing_kernel<<<(n + 255) / 256, 256, 0, s>>>(idx_in, w_in, n, k, E, idx, w, status);
  return cudaGetLastError();
}

}  // namespace moe
