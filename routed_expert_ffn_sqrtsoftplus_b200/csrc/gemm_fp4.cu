// Products of microscaled 4-bit matrices on tcgen05 block-scaled MMAs.
//
//   y[t, n] = xts * wts[g] * sum_k (x[t, k] 2^.. or sf) (w[g, n, k] 2^.. or sf)
//
// for one matrix (g = 0, all T rows), or one per expert: rows offsets[g] .. offsets[g + 1]
// of x meet w[g]. Both operands are E2M1, two values per byte in HBM and in shared memory;
// kind::mxf4 takes one E8M0 scale per 32 values of K, kind::mxf4nvf4 one E4M3 scale per 16.
//
// As in the layer's GEMMs the weights are the M operand (128 rows per MMA, kHalves MMAs
// sharing the token tile) and the tokens are N, so that one token still issues full-height
// MMAs and streams every weight byte once. Persistent CTAs, warp-specialised:
//   warp 0      TMA: a box of 256 values (128 bytes) x 128 kHalves rows of w, boxes of 32 rows of x
//   warp 1      copies a stage's scale factors to TMEM (tcgen05.cp) and issues its MMAs, four
//               K = 64 steps per ring stage
//   the others  epilogue, two or three per lane quarter taking interleaved 16-column chunks
//
// The MMA wants the scales of 128 rows as words of four K blocks, row r at 16 (r % 32) + 4 (r / 32),
// where HBM has rows of K / 32 or K / 16 bytes.
//   kPre = false (32-token tiles, bound by HBM): warp 14 brings a stage's scale rows into a ring of
//     their own (cp.async, 16 or 8 bytes a row, zeros outside), warps 2-5 turn them in place (lane l
//     takes rows l, l + 32, l + 64, l + 96). The weights' scales are read once, from where they are.
//   kPre = true (more tokens, bound by shared memory's bandwidth): a kernel in front arranges both
//     operands' scales into a workspace, and they come with the tiles, two bulk copies a stage.
//     Turned in the kernel they cost 24 KB of shared-memory traffic a stage by the LSUs, behind
//     MMAs that already read 107 of 128 bytes a cycle: turning a stage took 1000 to 3000 cycles
//     where its MMAs take 768.
//
// Measured (B200). NVFP4, 8192 x 4608 x 5120: 102 us with the scales' arrangement, 3.8 PFLOP/s, 4.1 where
// the tiles fill whole rounds (7872 rows), at the 1000 W cap (1.66 GHz); a stage of 256 x 192 takes 1075
// cycles of 768 of MMAs (940 without the TMA's writes: shared memory's bandwidth), a tile's epilogue 2500
// that the next tile does not cover. MXFP4, 384 experts of 5120 x 2304, 192 rows: 153 us, 6.1 TB/s of HBM;
// 64 experts of 2304 x 5120, 12288 rows: 125 us, of which 10 arrange 24 MB of scales. MXFP4, one row, 4608 x
// 5120: 8.1 us, of which 6.4 in the kernel: latencies of its first loads, seven stages, two cluster barriers.
//
// Few tokens and few tiles: a cluster of `splits` CTAs takes one tile, each a slice of K;
// the partial tiles meet in the first CTA's shared memory and are summed in slice order.
//
// Every read of offsets is clamped to [0, T] and to ascending order, so no offsets lead
// outside x or y. All waits are bounded; one that runs out makes its CTA give up, and the elements of y that it had
// not written yet stay as they were.
#include <cuda_fp16.h>

#include <atomic>

#include "common.cuh"
#include "kernels.h"

namespace moe {

namespace {

constexpr int kSfWarps = 4;
constexpr int kFirstSf = 2;
constexpr int kSfLoader = 14;
constexpr int kThreads = 32 * (kSfLoader + 1);
constexpr int kBK = 256;              // K values per stage
constexpr int kRowBytes = kBK / 2;    // 128: one swizzle row
constexpr int kBox = 32;              // token rows per TMA box
constexpr int kMaxExperts = 512;
constexpr int kMaxSplits = 8;
// Limit of the waits for a CTA's own copies and MMAs at its end, whatever the limit of the others: what is in flight
// then writes to memory that the CTA gives back.
constexpr uint64_t kDrainNs = 2000000000ull;

// kHalves: 128-row halves of w per tile; kBN: rows of x per tile.
template <bool kNv, bool kPre, int kHalves, int kBN>
struct Cfg {
  static constexpr int kABytes = kHalves * 128 * kRowBytes;
  static constexpr int kBBytes = kBN * kRowBytes;
  static constexpr int kTokens = kBN;
  static constexpr int kCols = 128 * kHalves;                      // rows of w, columns of y
  static constexpr int kFirstEpi = kPre ? kFirstSf : kFirstSf + kSfWarps;
  static constexpr int kEpiWarps = kPre ? 12 : 8;
  static constexpr int kEpiGroups = kEpiWarps / 4;
  static constexpr int kAtoms = kNv ? 4 : 2;                       // 32-bit words of scales per row and stage
  static constexpr int kBBlocks = (kBN + 127) / 128;               // 128-row blocks of x's scales
  static constexpr int kBCols = kBBlocks * 4;                      // TMEM columns of one word of them
  static constexpr int kSfCols = kAtoms * (4 * kHalves + kBCols);  // TMEM columns of one stage's scales
  static constexpr int kAccCols = kHalves * kBN;
  static constexpr int kAccs = 2 * kAccCols + 2 * kSfCols <= 512 ? 2 : 1;
  static constexpr int kSfBase = kAccs * kAccCols;
  static constexpr int kSets = kSfBase + 3 * kSfCols <= 512 ? 3 : 2;  // stages whose scales TMEM holds
  static constexpr int kRowSf = kNv ? 16 : 8;                      // scale bytes of a row and stage
  static constexpr int kBlocks = kHalves + kBBlocks;
  static constexpr int kBlockBytes = 128 * kRowSf;
  static constexpr int kRawBytes = kBlocks * kBlockBytes;
  static constexpr int kFixed = 1024 + 512 + 2 * (kMaxExperts + 1) * 4;  // alignment, barriers, experts
  // stages of scales in flight: as the tiles' where they come together, else six
  static constexpr int kFit = kPre ? (227 * 1024 - kFixed) / (kABytes + kBBytes + kRawBytes)
                                   : (227 * 1024 - kFixed - 6 * kRawBytes) / (kABytes + kBBytes);
  static constexpr int kStages = kFit > 8 ? 8 : kFit;
  static constexpr int kRaw = kPre ? kStages : 6;
  static constexpr int kSmemBytes = kFixed + kRaw * kRawBytes + kStages * (kABytes + kBBytes);
  static_assert(kSfBase + kSets * kSfCols <= 512 && kSets <= kRaw && kStages >= 2, "TMEM, ring");
  static_assert((2 * kStages + 3 * kRaw + 2 * kAccs + 1) * 8 + 16 <= 512, "barriers");
  // the partial tiles of a split fit in the ring (kHalves == 1, kBN == 32)
  static_assert(kHalves > 1 || kBN > 32 || (kMaxSplits - 1) * 128 * 32 * 4 <= kStages * (kABytes + kBBytes), "split");
};

// Instruction descriptor of the 4-bit kinds: E2M1 is format 1 (A bits 7-9, B bits 10-12), both
// K-major, N >> 3 in bits 17-22, scale format in bit 23 (1: E8M0, 0: E4M3), M >> 4 in bits 24-28,
// scale-factor ids in bits 4-5 (B) and 29-30 (A), both set by the caller, K = 64 (bit 31 = 0).
__device__ __forceinline__ uint32_t idesc_fp4(bool nv, uint32_t N) {
  return (1u << 7) | (1u << 10) | ((N >> 3) << 17) | ((nv ? 0u : 1u) << 23) | ((128u >> 4) << 24);
}

// True in one lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}\n" : "=r"(p));
  return p != 0;
}

// The descriptors' high halves (layout, strides) are the same everywhere; the low ones hold the
// address.
template <bool kNv>
__device__ __forceinline__ void umma_fp4(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t hi, uint32_t idesc,
                                         uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
  if constexpr (kNv)
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "mov.b64 a, {%1, %3};\n\tmov.b64 b, {%2, %3};\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], a, b, %4, [%6], [%7], p;\n\t}\n" ::
            "r"(d),
        "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "mov.b64 a, {%1, %3};\n\tmov.b64 b, {%2, %3};\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], a, b, %4, [%6], [%7], p;\n\t}\n" ::"r"(d),
        "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb)
        : "memory");
}
// tmem_cp_32x128b_x4 with the descriptor in halves.
__device__ __forceinline__ void copy_word(uint32_t taddr, uint32_t lo, uint32_t hi) {
  asm volatile(
      "{\n\t.reg .b64 s;\n\tmov.b64 s, {%1, %2};\n\ttcgen05.cp.cta_group::1.32x128b.warpx4 [%0], s;\n\t}\n" ::"r"(
          taddr),
      "r"(lo), "r"(hi)
      : "memory");
}

__device__ __forceinline__ uint32_t cluster_ctarank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Store to the same shared-memory address of another CTA of the cluster.
__device__ __forceinline__ void st_cluster_u32(uint32_t saddr, uint32_t rank, uint32_t v) {
  asm volatile(
      "{\n\t.reg .b32 a;\n\t"
      "mapa.shared::cluster.u32 a, %0, %1;\n\t"
      "st.shared::cluster.u32 [a], %2;\n\t}\n" ::"r"(saddr),
      "r"(rank), "r"(v)
      : "memory");
}

// Where a wait that ran out is recorded when the caller gave no word for it: one per device, for all its calls.
__device__ int product_status;
__device__ __forceinline__ void report_timeout(int* status) {
  report_status(status != nullptr ? status : &product_status, kStatusTimeout);
}

// mbarrier.try_wait that may suspend the thread for up to 20 us (it wakes when the phase completes).
__device__ __forceinline__ bool try_wait_suspended(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 20000;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
// The slow path of a wait, kept out of line: the roles' loops have to stay small (their warps share
// the SM's instruction caches).
__device__ __noinline__ bool wait_longer(uint64_t* bar, uint32_t parity, unsigned long long timeout_ns, int* status,
                                         volatile int* abort_flag) {
  const uint64_t t0 = globaltimer_ns();
  // a short wait polls (a suspended thread wakes some 300 ns late); a long one, a whole tile's say,
  // stays out of the way of the MMAs' reads of shared memory
#pragma unroll 1
  for (int i = 0; i < 64; ++i)
    if (mbar_try_wait(bar, parity)) return true;
  while (true) {
    if (try_wait_suspended(bar, parity)) return true;
    if (*abort_flag) return false;
    if (globaltimer_ns() - t0 > timeout_ns) {
      *abort_flag = 1;
      report_timeout(status);
      return false;
    }
  }
}
__device__ __forceinline__ bool wait_or_abort(uint64_t* bar, uint32_t parity, const Fp4GemmArgs& a,
                                              volatile int* abort_flag) {
  return mbar_try_wait(bar, parity) || wait_longer(bar, parity, a.timeout_ns, a.status, abort_flag);
}
// The same by a whole converged warp, which leaves it together: the loop branches on votes alone and
// calls nothing, so that the code around it keeps its addresses in uniform registers.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, unsigned long long timeout_ns) {
  uint64_t t0 = 0;
  for (uint32_t i = 0; !__all_sync(0xffffffffu, mbar_try_wait(bar, parity)); ++i) {
    if ((i & 255u) == 255u) {
      const uint64_t now = globaltimer_ns();
      if (t0 == 0) t0 = now;
      if (__any_sync(0xffffffffu, now - t0 > timeout_ns)) return false;
    }
  }
  return true;
}

// Waits until the last `stages` of a ring's copies issued so far have landed.
__device__ __noinline__ void drain_ring(uint64_t* full, int stages, long issued) {
  for (long i = issued - 1; i >= 0 && i >= issued - stages; --i) {
    const uint64_t b = globaltimer_ns();
    while (!mbar_try_wait(&full[i % stages], static_cast<uint32_t>((i / stages) & 1)) && globaltimer_ns() - b < kDrainNs) {
    }
  }
}

// A value that is the same in all lanes, into a uniform register.
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __reduce_or_sync(0xffffffffu, v); }

struct Tile {
  int g;           // expert
  int row0, rows;  // tokens
  int col0, cols;  // rows of w[g]
  int xtile, wtile;  // number of the token tile and of the w tile
};

// Tile t: experts in order, inside an expert the w tiles in order, inside a w tile its token
// tiles, so that CTAs taking consecutive tiles read the same weights together, through L2.
// `pre` holds each expert's first token tile, `row` its first row.
template <int kTokens, int kCols>
__device__ __noinline__ Tile tile_of_(int t, int E, int N, int m_tiles, const int* pre, const int* row) {
  int lo = 0, hi = E - 1;
  const int want = t / m_tiles;  // pre[g] * m_tiles <= t  <=>  pre[g] <= t / m_tiles
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (pre[mid] <= want) lo = mid; else hi = mid - 1;
  }
  const int nt = pre[lo + 1] - pre[lo];
  const int local = t - pre[lo] * m_tiles;
  const int m = local / nt, n = local - m * nt;
  Tile r;
  r.g = lo;
  r.row0 = row[lo] + n * kTokens;
  r.rows = min(kTokens, row[lo + 1] - r.row0);
  r.col0 = m * kCols;
  r.cols = min(kCols, N - r.col0);
  r.xtile = pre[lo] + n;
  r.wtile = lo * m_tiles + m;
  return r;
}
template <class C>
__device__ __forceinline__ Tile tile_of(int t, const Fp4GemmArgs& a, const int* pre, const int* row) {
  return tile_of_<C::kTokens, C::kCols>(t, a.E, a.N, a.m_tiles, pre, row);
}

// The experts' rows and token tiles, by one warp, 32 experts at a time: row[g] the first row of expert
// g (clamped to [0, T] and to ascending order), pre[g] its first token tile, g = 0 .. E.
template <int kTokens>
__device__ __forceinline__ void scan_experts(const int32_t* offsets, int E, int T, int* pre, int* row) {
  const int lane = threadIdx.x % 32;
  int last = 0, tiles = 0;
  for (int b = 0; b <= E; b += 32) {
    const int g = b + lane;
    int v = 0;
    if (g <= E) v = offsets ? max(0, min(T, __ldg(offsets + g))) : (g == 0 ? 0 : T);
    // running maximum: offsets that go back leave an expert without rows
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v = max(v, u);
    }
    v = max(v, last);
    int before = __shfl_up_sync(0xffffffffu, v, 1);
    if (lane == 0) before = last;
    // token tiles of expert g - 1 end at g
    int n = g > 0 && g <= E ? (v - before + kTokens - 1) / kTokens : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, n, o);
      if (lane >= o) n += u;
    }
    if (g <= E) {
      row[g] = v;
      pre[g] = tiles + n;
    }
    tiles += __shfl_sync(0xffffffffu, n, 31);
    last = __shfl_sync(0xffffffffu, v, 31);
  }
}

// kBytes (8 or 16) to shared memory, the first n of them from global memory, zeros behind.
template <int kBytes>
__device__ __forceinline__ void cp_async_zfill(uint32_t dst, const void* src, int n) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(src)),
               "n"(kBytes), "r"(n)
               : "memory");
}
// Arrive on bar once this thread's copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// A row's kWords scale words of a stage, from shared memory.
template <int kWords>
__device__ __forceinline__ void read_scales(const uint8_t* p, uint32_t* w) {
  if constexpr (kWords == 4) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    w[0] = v.x;
    w[1] = v.y;
    w[2] = v.z;
    w[3] = v.w;
  } else {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x;
    w[1] = v.y;
  }
}

__device__ __forceinline__ uint32_t pack_pair(bool bf, float lo, float hi) {
  if (bf) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// 16 tokens of output column n = this lane's row of w, as 16-bit pairs (token 2j low, 2j + 1 high).
// vec: four lanes exchange theirs so that each holds four consecutive columns of a token, and a warp
// stores 64 bytes of four tokens at a time instead of 64 bytes of one (8 shuffles and 4 stores for
// 16 stores); N % 4 == 0 keeps a group of four on one side of N.
__device__ __forceinline__ void store_pairs(const Fp4GemmArgs& a, int row0, int c0, int nrows, int n, int lane,
                                            bool vec, const uint32_t (&p)[8]) {
  uint16_t* out = static_cast<uint16_t*>(a.out) + static_cast<int64_t>(row0 + c0) * a.N;
  if (vec) {
    const bool odd = lane & 1, up = lane & 2;
    uint32_t q[8];  // q[m]: token 2m + odd, columns n & ~1 and the next
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t lo = __byte_perm(p[2 * i], p[2 * i + 1], 0x5410), hi = __byte_perm(p[2 * i], p[2 * i + 1], 0x7632);
      const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? lo : hi, 1);
      const uint32_t l = odd ? got : lo, r = odd ? hi : got;
      q[2 * i] = __byte_perm(l, r, 0x5410);
      q[2 * i + 1] = __byte_perm(l, r, 0x7632);
    }
    const int token = lane & 3;
    uint16_t* dst = out + static_cast<int64_t>(token) * a.N + (n & ~3);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t keep = up ? q[2 * i + 1] : q[2 * i];
      const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? q[2 * i] : q[2 * i + 1], 2);
      if (n < a.N && c0 + 4 * i + token < nrows)
        *reinterpret_cast<uint2*>(dst) = up ? make_uint2(got, keep) : make_uint2(keep, got);
      dst += 4 * static_cast<int64_t>(a.N);
    }
    return;
  }
  if (n >= a.N) return;
#pragma unroll
  for (int j = 0; j < 16; ++j)
    if (c0 + j < nrows)
      out[static_cast<int64_t>(j) * a.N + n] = static_cast<uint16_t>(p[j / 2] >> (16 * (j & 1)));
}

// The two tensor scales as (first, then) factors of an accumulator. Their product alone (first = 1) where it is a
// normal number. Two scales far apart from 1 may multiply to none although the results are: accumulators are 0 or
// between 2^-20 (half times half, with the least scales) and 2^41, so 2^-+80 times the product's mantissa keeps them
// normal numbers, and the rest is a power of two, cut off where every result is 0 or infinite.
__device__ __noinline__ float2 far_scales(float xts, float wts) {
  if (!(fabsf(xts) < INFINITY && fabsf(wts) < INFINITY)) return make_float2(1.0f, xts * wts);
  int ex, ew;
  const float f = frexpf(xts, &ex) * frexpf(wts, &ew);
  const int e = ex + ew;
  return e < 0 ? make_float2(f * 0x1p-80f, ldexpf(1.0f, max(e + 80, -126)))
               : make_float2(f * 0x1p80f, ldexpf(1.0f, min(e - 80, 127)));
}
__device__ __forceinline__ float2 tensor_scales(float xts, float wts) {
  const float m = xts * wts;
  return fabsf(m) >= 0x1p-126f && fabsf(m) < INFINITY ? make_float2(1.0f, m) : far_scales(xts, wts);
}
__device__ __forceinline__ void scale_16(uint32_t (&r)[16], float first) {
#pragma unroll
  for (int j = 0; j < 16; ++j) r[j] = __float_as_uint(first * __uint_as_float(r[j]));
}

// 16 accumulator columns (tokens) scaled and rounded to 16 bits, as pairs.
__device__ __forceinline__ void pack_16(bool bf, float alpha, const uint32_t (&r)[16], uint32_t (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j)
    v[j] = pack_pair(bf, alpha * __uint_as_float(r[2 * j]), alpha * __uint_as_float(r[2 * j + 1]));
}
// The same in 32 bits, stored: tokens c0 .. c0 + 15 of row m of the tile.
__device__ __forceinline__ void store_f32(const Fp4GemmArgs& a, const Tile& tl, int m, int c0, float alpha,
                                          const uint32_t (&r)[16]) {
  if (m >= tl.cols) return;
  float* p = static_cast<float*>(a.out) + static_cast<int64_t>(tl.row0 + c0) * a.N + tl.col0 + m;
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    if (c0 + j < tl.rows) *p = alpha * __uint_as_float(r[j]);
    p += a.N;
  }
}

// The same in either width for scales with a factor that comes first, from TMEM. Out of line and with plain arguments:
// a test of that factor in the 16-bit path costs it 1 %, a reference to the kernel's arguments 4 %.
__device__ __noinline__ void store_far(void* out, int out_dtype, int N, uint32_t taddr, int row0, int n, int nrows,
                                       float first, float alpha) {
  uint32_t r[16];
  tmem_ld16(taddr, r);
  tmem_ld_wait();
  if (n >= N) return;
  scale_16(r, first);
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    if (j >= nrows) break;
    const float v = alpha * __uint_as_float(r[j]);
    const int64_t at = static_cast<int64_t>(row0 + j) * N + n;
    if (out_dtype == kValFp32) static_cast<float*>(out)[at] = v;
    else static_cast<uint16_t*>(out)[at] = static_cast<uint16_t>(pack_pair(out_dtype == kValBf16, v, 0.0f));
  }
}

template <bool kNv, bool kPre, int kHalves, int kBN, bool kSplit>
__global__ void __launch_bounds__(kThreads, 1)
    gemm_fp4_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                    const Fp4GemmArgs args) {
  using C = Cfg<kNv, kPre, kHalves, kBN>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sA = smem;
  uint8_t* sB = sA + C::kStages * C::kABytes;
  uint8_t* sRaw = sB + C::kStages * C::kBBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sRaw + C::kRaw * C::kRawBytes);
  uint64_t* full = bars;
  uint64_t* empty = full + C::kStages;
  uint64_t* tfull = empty + C::kStages;
  uint64_t* tempty = tfull + C::kAccs;
  uint64_t* rfull = tempty + C::kAccs;   // scale rows landed
  uint64_t* rturned = rfull + C::kRaw;   // ... and put in the MMA's order
  uint64_t* rempty = rturned + C::kRaw;
  uint64_t* drain = rempty + C::kRaw;
  uint32_t* tmem_base_smem = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_base_smem + 1);
  volatile long* issued_s = reinterpret_cast<volatile long*>(tmem_base_smem + 2);  // stages that the producer issued
  int* pre = reinterpret_cast<int*>(reinterpret_cast<uint8_t*>(bars) + 512);  // [E + 1] first token tile
  int* row_s = pre + kMaxExperts + 1;                                         // [E + 1] first row

  const int warp = threadIdx.x / 32;
  const int lane = threadIdx.x % 32;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < C::kRaw; ++i) {
      mbar_init(&rfull[i], 32);
      mbar_init(&rturned[i], kSfWarps);
      mbar_init(&rempty[i], 1);
    }
    for (int i = 0; i < C::kAccs; ++i) {
      mbar_init(&tfull[i], 1);
      mbar_init(&tempty[i], C::kEpiWarps);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbarrier_init();
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
  }
  // everything above overlaps a quantiser of few blocks in front (the scales' arrangement lets no kernel start early);
  // TMEM is taken behind it, so that no block waits for a kernel that waits for this block's columns
  wait_for_previous_kernel();
  if (warp == 1) {
    tmem_alloc(tmem_base_smem, 512);
    tmem_relinquish();
  }
  if (warp == kFirstSf) scan_experts<C::kTokens>(args.offsets, args.E, args.T, pre, row_s);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_base_smem;
  // a loop bound that came from memory would make the compiler treat the MMA warp's loop as divergent:
  // each tcgen05 instruction then costs some 35 cycles of moves into uniform registers instead of 8
  const int total = static_cast<int>(uniform(static_cast<uint32_t>(pre[args.E] * args.m_tiles)));

  // split: one tile per cluster, K cut into `splits` slices; otherwise a strided list of tiles
  const int rank = kSplit ? static_cast<int>(cluster_ctarank()) : 0;
  const int splits = kSplit ? args.splits : 1;
  const int t0 = static_cast<int>(blockIdx.x) / splits;
  const int stride = kSplit ? 0x40000000 : static_cast<int>(gridDim.x);
  const int kb0 = kSplit ? args.num_kb * rank / splits : 0;
  const int kb1 = kSplit ? args.num_kb * (rank + 1) / splits : args.num_kb;

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      long issued = 0;
      for (int t = t0; t < total && !*abort_flag; t += stride) {
        const Tile tl = tile_of<C>(t, args, pre, row_s);
        const int w_row = tl.g * args.N + tl.col0;
        const int nb = (tl.rows + kBox - 1) / kBox;
        // weights that one token tile alone reads stream past; what many tiles read stays in L2
        constexpr uint64_t w_hint = kBN >= 192 ? kCacheEvictNormal : kCacheEvictFirst;
        bool ok = true;
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!wait_or_abort(&empty[stage], phase ^ 1, args, abort_flag)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&full[stage], C::kABytes + nb * kBox * kRowBytes + (kPre ? C::kRawBytes : 0));
          tma_load_2d(sA + stage * C::kABytes, &tmA, &full[stage], kb * kRowBytes, w_row, w_hint);
          for (int j = 0; j < nb; ++j)
            tma_load_2d(sB + stage * C::kBBytes + j * kBox * kRowBytes, &tmB, &full[stage], kb * kRowBytes,
                        tl.row0 + j * kBox, kCacheEvictLast);
          if constexpr (kPre) {
            constexpr int kWSf = kHalves * C::kAtoms * 512, kXSf = C::kBBlocks * C::kAtoms * 512;
            const int64_t wt = static_cast<int64_t>(tl.wtile) * args.num_kb + kb;
            const int64_t xt = static_cast<int64_t>(tl.xtile) * args.num_kb + kb;
            uint8_t* sf = sRaw + stage * C::kRawBytes;
            bulk_load(sf, args.ws_tiles + wt * kWSf, kWSf, &full[stage], kCacheEvictNormal);
            bulk_load(sf + kWSf, args.xs_tiles + xt * kXSf, kXSf, &full[stage],
                      kCacheEvictNormal);
          }
          ++issued;
          if (++stage == C::kStages) {
            stage = 0;
            phase ^= 1;
          }
        }
        if (!ok) break;
      }
      *issued_s = issued;
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    // The whole warp walks the stages and agrees on every wait, so that the loop and its addresses
    // are the same in all lanes (uniform registers); one elected lane issues. With the loop inside
    // `lane == 0` a tcgen05 instruction took some 80 cycles to issue, with waits that each lane
    // judged by itself 57.
    //
    // kPre: the copies of the next stage's scales go ahead of a stage's last MMAs. Copies issued ahead of
    // a stage's own first MMAs leave the tensor core idle, and the columns they go to are free only
    // once the stage before this one is through.
    const bool elected = elect_one();
    const uint32_t tmem = uniform(tmem_base);
    const uint64_t tile_desc = sdesc_sw128(smem_u32(sA)), raw_desc = sdesc_plain(smem_u32(sRaw));
    const uint32_t a_lo0 = static_cast<uint32_t>(tile_desc), hi = static_cast<uint32_t>(tile_desc >> 32);
    const uint32_t b_lo0 = static_cast<uint32_t>(sdesc_sw128(smem_u32(sB)));
    const uint32_t raw_lo0 = static_cast<uint32_t>(raw_desc), raw_hi = static_cast<uint32_t>(raw_desc >> 32);
    int stage = 0, raw = 0, set = 0, acc = 0;
    uint32_t phase = 0, rphase = 0, aphase = 0;
    int old = 0;       // scale slot of the stage that used the next set of TMEM columns before
    uint32_t ophase = 0;
    int n_stage = 1;   // stages whose scales were copied so far, up to kSets
    // blocks [b0, b1) of the scales in slot ra, to the columns of set se
    auto copy_scales = [&](int ra, int se, int b0, int b1) {
      const uint32_t sf = tmem + C::kSfBase + se * C::kSfCols;
      const uint32_t lo = raw_lo0 + static_cast<uint32_t>(ra * (C::kRawBytes / 16));
#pragma unroll
      for (int b = 0; b < C::kBlocks; ++b)
        if (b >= b0 && b < b1)
#pragma unroll
          for (int j = 0; j < C::kAtoms; ++j)
            copy_word(sf + (b < kHalves ? (b * C::kAtoms + j) * 4
                                        : kHalves * C::kAtoms * 4 + j * C::kBCols + (b - kHalves) * 4),
                      lo + (b * C::kBlockBytes + j * 512) / 16, raw_hi);
    };
    bool ok = true;
    if (kPre && t0 < total) {
      ok = warp_wait(&full[0], 0, args.timeout_ns);
      tc_fence_after();
      if (elected) copy_scales(0, 0, 0, C::kBlocks);
      __syncwarp();
    }
    // waits until the MMAs that last read the next set of TMEM columns are done: their scales' slot
    // is free then (kSets <= kRaw: its barrier cannot have moved on by a second phase)
    auto set_free = [&]() {
      uint64_t* slot = kPre ? empty : rempty;
      if (n_stage < C::kSets) {
        ++n_stage;
        return true;
      }
      const bool w = warp_wait(&slot[old], ophase, args.timeout_ns);
      if (++old == C::kRaw) {
        old = 0;
        ophase ^= 1;
      }
      return w;
    };
    for (int t = t0; ok && t < total; t += stride) {
      const Tile tl = tile_of<C>(t, args, pre, row_s);
      const uint32_t n_mma = (tl.rows + 15) & ~15;
      const uint32_t idesc = uniform(idesc_fp4(kNv, n_mma));
      ok = warp_wait(&tempty[acc], aphase ^ 1, args.timeout_ns);
      if (!ok) break;
      tc_fence_after();
      const uint32_t d = tmem + acc * C::kAccCols;
      for (int kb = kb0; kb < kb1; ++kb) {
        const uint32_t sf = tmem + C::kSfBase + set * C::kSfCols;
        const uint32_t a_lo = a_lo0 + static_cast<uint32_t>(stage * (C::kABytes / 16));
        const uint32_t b_lo = b_lo0 + static_cast<uint32_t>(stage * (C::kBBytes / 16));
        const uint32_t first = kb != kb0;
        auto mma_step = [&](uint32_t j, uint32_t accumulate) {
          const uint32_t atom = kNv ? j : j / 2, id = kNv ? 0 : (j & 1) * 2;
#pragma unroll
          for (uint32_t h = 0; h < kHalves; ++h)
            umma_fp4<kNv>(d + h * kBN, a_lo + (h * 128 * kRowBytes + j * 32) / 16, b_lo + j * 2, hi,
                          idesc | (id << 4) | (id << 29), (sf + (h * C::kAtoms + atom) * 4) | (id << 30),
                          (sf + kHalves * C::kAtoms * 4 + atom * C::kBCols) | (id << 30), accumulate);
        };
        if constexpr (kPre) {
          // this stage arrived with the last one's wait
          if (elected) {
            mma_step(0, first);
            mma_step(1, 1u);
            mma_step(2, 1u);
          }
          __syncwarp();
          const int nstage = stage + 1 == C::kStages ? 0 : stage + 1;
          const uint32_t nphase = stage + 1 == C::kStages ? phase ^ 1 : phase;
          const int nset = set + 1 == C::kSets ? 0 : set + 1;
          if (kb + 1 < kb1 || t + stride < total) ok = warp_wait(&full[nstage], nphase, args.timeout_ns);
          ok = ok && set_free();
          if (!ok) break;
          tc_fence_after();
          // no branch in here: behind the last stage of all, the copies bring what nothing reads, to
          // columns that nothing reads any more
          // (with the copies under a condition the compiler gave up the uniform registers of the whole
          // region, and a stage took 1510 cycles instead of 920)
          if (elected) {
            copy_scales(nstage, nset, 0, C::kBlocks);
            mma_step(3, 1u);
            umma_commit(&empty[stage]);
          }
          __syncwarp();
          stage = nstage;
          phase = nphase;
          set = nset;
        } else {
          ok = warp_wait(&rturned[raw], rphase, args.timeout_ns) && (kb == kb0 && t == t0 ? true : set_free()) &&
               warp_wait(&full[stage], phase, args.timeout_ns);
          if (!ok) break;
          tc_fence_after();
          if (elected) {
            copy_scales(raw, set, 0, C::kBlocks);
            mma_step(0, first);
            mma_step(1, 1u);
            mma_step(2, 1u);
            mma_step(3, 1u);
            umma_commit(&empty[stage]);
            umma_commit(&rempty[raw]);
          }
          __syncwarp();
          if (++stage == C::kStages) {
            stage = 0;
            phase ^= 1;
          }
          if (++raw == C::kRaw) {
            raw = 0;
            rphase ^= 1;
          }
          if (++set == C::kSets) set = 0;
        }
      }
      if (!ok) break;
      if (elected) umma_commit(&tfull[acc]);
      __syncwarp();
      if (++acc == C::kAccs) {
        acc = 0;
        aphase ^= 1;
      }
    }
    if (!ok && elected) {
      *abort_flag = 1;
      report_timeout(args.status);
    }
    // every MMA done before TMEM and shared memory go
    if (elected) {
      umma_commit(drain);
      const uint64_t b = globaltimer_ns();
      while (!mbar_try_wait(drain, 0) && globaltimer_ns() - b < kDrainNs) {
      }
    }
    __syncwarp();
  } else if (!kPre && warp < C::kFirstEpi) {
    // ------------------------------------------------------------ scale rows -> the MMA's order
    constexpr int kW = C::kAtoms;
    int raw = 0;
    uint32_t rphase = 0;
    bool ok = true;
    for (int t = t0; ok && t < total; t += stride) {
      for (int kb = kb0; kb < kb1; ++kb) {
        if (lane == 0) ok = wait_or_abort(&rfull[raw], rphase, args, abort_flag);
        ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
        if (!ok) break;
        for (int b = warp - kFirstSf; b < C::kBlocks; b += kSfWarps) {
          uint8_t* block = sRaw + raw * C::kRawBytes + b * C::kBlockBytes;
          uint32_t w[4 * kW];
#pragma unroll
          for (int i = 0; i < 4; ++i) read_scales<kW>(block + (32 * i + lane) * C::kRowSf, w + i * kW);
          __syncwarp();  // every row is read before any column is written
#pragma unroll
          for (int j = 0; j < kW; ++j)
            *reinterpret_cast<uint4*>(block + j * 512 + lane * 16) =
                make_uint4(w[j], w[kW + j], w[2 * kW + j], w[3 * kW + j]);
        }
        fence_proxy_async_smem();  // the tensor core reads what these generic stores wrote
        __syncwarp();
        if (lane == 0) mbar_arrive(&rturned[raw]);
        if (++raw == C::kRaw) {
          raw = 0;
          rphase ^= 1;
        }
      }
    }
  } else if (!kPre && warp == kSfLoader) {
    // ------------------------------------------------------------ scale rows -> shared memory
    constexpr int kB = C::kRowSf;
    int raw = 0;
    uint32_t rphase = 0;
    bool ok = true;
    const int64_t w_step = 32 * args.ws_stride, x_step = 32 * args.xs_stride;
    for (int t = t0; ok && t < total; t += stride) {
      const Tile tl = tile_of<C>(t, args, pre, row_s);
      const uint8_t* wrow = args.ws + (static_cast<int64_t>(tl.g) * args.N + tl.col0 + lane) * args.ws_stride;
      const uint8_t* xrow = args.xs + static_cast<int64_t>(tl.row0 + lane) * args.xs_stride;
      const int w_left = tl.cols - lane, x_left = tl.rows - lane;  // rows from this lane's first one
      for (int kb = kb0; kb < kb1; ++kb) {
        if (lane == 0) ok = wait_or_abort(&rempty[raw], rphase ^ 1, args, abort_flag);
        ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
        if (!ok) break;
        const uint32_t dst = smem_u32(sRaw + raw * C::kRawBytes + lane * kB);
        const int off = kb * kB;
        const int left = min(kB, args.sf_cols - off);
        const uint8_t* pw = wrow + off;
        const uint8_t* px = xrow + off;
        // a row outside reads nothing (0 bytes from the scales' own start)
#pragma unroll
        for (int i = 0; i < 4 * kHalves; ++i) {
          const bool in = 32 * i < w_left;
          cp_async_zfill<kB>(dst + i * 32 * kB, in ? pw : args.ws, in ? left : 0);
          pw += w_step;
        }
#pragma unroll
        for (int i = 0; i < kBN / 32; ++i) {
          const bool in = 32 * i < x_left;
          cp_async_zfill<kB>(dst + (4 * kHalves + i) * 32 * kB, in ? px : args.ws, in ? left : 0);
          px += x_step;
        }
        cp_async_arrive(&rfull[raw]);
        if (++raw == C::kRaw) {
          raw = 0;
          rphase ^= 1;
        }
      }
    }
    // copies in flight land before the CTA's shared memory goes
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (warp >= C::kFirstEpi && warp < kSfLoader) {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3;
    const int cfirst = ((warp - C::kFirstEpi) / 4) * 16;
    const float xts = args.x_ts ? __ldg(args.x_ts) : 1.0f;
    const bool vec_out = args.N % 4 == 0 && (reinterpret_cast<uintptr_t>(args.out) & 7) == 0;
    int acc = 0;
    uint32_t aphase = 0;
    for (int t = t0; t < total; t += stride) {
      const Tile tl = tile_of<C>(t, args, pre, row_s);
      bool ok = true;
      if (lane == 0) ok = wait_or_abort(&tfull[acc], aphase, args, abort_flag);
      ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
      if (!ok) break;
      tc_fence_after();
      if constexpr (!kSplit) {
        const float2 scales = args.w_ts ? tensor_scales(xts, __ldg(args.w_ts + tl.g)) : make_float2(1.0f, xts);
        const float alpha = scales.y;
        const uint32_t tb = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + acc * C::kAccCols;
        const int mine = q * 32 + lane;  // this lane's row of the tile's first half
        if (scales.x != 1.0f) {
          for (int c0 = cfirst; c0 < tl.rows; c0 += 16 * C::kEpiGroups)
            for (int h = 0; h < kHalves; ++h)
              store_far(args.out, args.out_dtype, args.N, tb + h * kBN + c0, tl.row0 + c0, tl.col0 + mine + h * 128,
                        tl.rows - c0, scales.x, scales.y);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&tempty[acc]);
        } else if (args.out_dtype == kValFp32) {
#pragma unroll 1
          for (int c0 = cfirst; c0 < tl.rows; c0 += 16 * C::kEpiGroups) {
#pragma unroll
            for (int h = 0; h < kHalves; ++h) {  // (as a loop it cost 142 to 147 us, by its place, instead of 139: 8192 x 4608 x 5120)
              uint32_t r[16];
              tmem_ld16(tb + h * kBN + c0, r);
              tmem_ld_wait();
              store_f32(args, tl, mine + h * 128, c0, alpha, r);
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&tempty[acc]);
        } else {
          // 16-bit results fit in registers as pairs: take the whole tile out of TMEM, give it back to
          // the MMAs, and store while the next tile's run
          constexpr int kChunks = (kBN / 16 + C::kEpiGroups - 1) / C::kEpiGroups;
          const bool bf = args.out_dtype == kValBf16;
          uint32_t hold[kChunks][kHalves][8];
#pragma unroll
          for (int i = 0; i < kChunks; ++i) {
            const int c0 = cfirst + i * 16 * C::kEpiGroups;
            if (c0 < tl.rows) {
              uint32_t r[kHalves][16];
#pragma unroll
              for (int h = 0; h < kHalves; ++h) tmem_ld16(tb + h * kBN + c0, r[h]);
              tmem_ld_wait();
#pragma unroll
              for (int h = 0; h < kHalves; ++h) pack_16(bf, alpha, r[h], hold[i][h]);
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&tempty[acc]);
#pragma unroll
          for (int i = 0; i < kChunks; ++i) {
            const int c0 = cfirst + i * 16 * C::kEpiGroups;
            if (c0 < tl.rows) {
#pragma unroll
              for (int h = 0; h < kHalves; ++h)
                store_pairs(args, tl.row0, c0, tl.rows, tl.col0 + mine + h * 128, lane, vec_out, hold[i][h]);
            }
          }
        }
      }
      if (++acc == C::kAccs) {
        acc = 0;
        aphase ^= 1;
      }
    }
  }

  if constexpr (kSplit) {
    // every CTA of the cluster is through its slice: the first one's ring is free for the
    // others' partial tiles, [slice - 1][token][128]
    __syncthreads();
    cluster_sync_all();
    const int q = warp & 3;
    const int cfirst = ((warp - C::kFirstEpi) / 4) * 16;
    const bool work = warp >= C::kFirstEpi && warp < kSfLoader && t0 < total && !*abort_flag;
    Tile tl{};
    if (work) tl = tile_of<C>(t0, args, pre, row_s);
    uint32_t r[16];
    if (work && cfirst < tl.rows) {
      tc_fence_after();
      tmem_ld16(tmem_base + (static_cast<uint32_t>(q * 32) << 16) + cfirst, r);
      tmem_ld_wait();
      if (rank != 0) {
        const uint32_t dst = smem_u32(sA) + (((rank - 1) * kBN + cfirst) * 128 + q * 32 + lane) * 4;
#pragma unroll
        for (int j = 0; j < 16; ++j) st_cluster_u32(dst + j * 512, 0, r[j]);
      }
    }
    // a CTA that gave up has no part to add: the first one then writes nothing
    if (threadIdx.x == 0 && rank != 0 && *abort_flag) st_cluster_u32(smem_u32(const_cast<int*>(abort_flag)), 0, 1u);
    __syncwarp();
    cluster_sync_all();
    if (work && rank == 0 && !*abort_flag && cfirst < tl.rows) {
      const float* part = reinterpret_cast<const float*>(sA) + cfirst * 128 + q * 32 + lane;
      for (int p = 0; p < splits - 1; ++p)
#pragma unroll
        for (int j = 0; j < 16; ++j)
          r[j] = __float_as_uint(__uint_as_float(r[j]) + part[(p * kBN + j) * 128]);
      const float xts = args.x_ts ? __ldg(args.x_ts) : 1.0f;
      const float2 scales = args.w_ts ? tensor_scales(xts, __ldg(args.w_ts + tl.g)) : make_float2(1.0f, xts);
      const float alpha = scales.y;
      if (scales.x != 1.0f) scale_16(r, scales.x);
      const int m = q * 32 + lane;
      const bool vec_out = args.N % 4 == 0 && (reinterpret_cast<uintptr_t>(args.out) & 7) == 0;
      if (args.out_dtype == kValFp32) {
        store_f32(args, tl, m, cfirst, alpha, r);
      } else {
        uint32_t v[8];
        pack_16(args.out_dtype == kValBf16, alpha, r, v);
        store_pairs(args, tl.row0, cfirst, tl.rows, tl.col0 + m, lane, vec_out, v);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  // where the CTA gave up, whichever warp did and when: its copies land before its shared memory goes (asked here, as the
  // producer may be through before another warp gives up)
  if (threadIdx.x == 0 && *abort_flag) drain_ring(full, C::kStages, *issued_s);
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, 512);
  }
}

template <bool kNv, bool kPre, int kHalves, int kBN, bool kSplit>
cudaError_t launch_cfg(const CUtensorMap& tw, const CUtensorMap& tx, const Fp4GemmArgs& a, int grid, cudaStream_t s) {
  using C = Cfg<kNv, kPre, kHalves, kBN>;
  auto* kernel = gemm_fp4_kernel<kNv, kPre, kHalves, kBN, kSplit>;
  // the kernel's shared memory, allowed once per device
  static std::atomic<uint64_t> allowed{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !((allowed.load(std::memory_order_relaxed) >> dev) & 1)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
    if (e != cudaSuccess) return e;
    if (dev < 64) allowed.fetch_or(uint64_t(1) << dev, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::kSmemBytes;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = kSplit ? a.splits : 1;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = kSplit ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, tw, tx, a);
}

// Scales into the MMA's order: for each tile (of kCols rows of w, or of kTokens rows of x) and each K
// block of 256, 128-row blocks of kNv ? 4 : 2 words, each word 512 bytes with row r at 16 (r % 32) +
// 4 (r / 32); zeros for rows outside the tile and behind a row's end. Blocks x: the tiles of w, expert
// by expert, then those of x; y: 64 bytes of every row. A thread takes 16 bytes of rows l, l + 32, l + 64
// and l + 96, a neighbour the next 16: a 4 x 4 matrix of words, whose columns are the 16-byte pieces.
constexpr int kArrangeBytes = 64;
// A row's 16 bytes at c, zeros from n on.
__device__ __forceinline__ uint4 scale_words(const uint8_t* row, int c, int n, int align) {
  const uint8_t* s = row + c;
  if (align >= 16 && c + 16 <= n) return __ldg(reinterpret_cast<const uint4*>(s));
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    w[j] = 0u;
    if (align >= 4 && c + 4 * j + 4 <= n) {
      w[j] = __ldg(reinterpret_cast<const uint32_t*>(s + 4 * j));
    } else {
      for (int e = 0; e < 4; ++e)
        if (c + 4 * j + e < n) w[j] |= static_cast<uint32_t>(__ldg(s + 4 * j + e)) << (8 * e);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
template <bool kNv, int kRows>
__device__ __forceinline__ void arrange_tile(const uint8_t* src, int64_t stride, int rows, int sf_cols, int num_kb,
                                             uint4* out) {
  constexpr int kWords = kNv ? 4 : 2, kBlocks = (kRows + 127) / 128;
  const uint64_t at = reinterpret_cast<uintptr_t>(src) | static_cast<uint64_t>(stride);
  const int align = at % 16 == 0 ? 16 : at % 4 == 0 ? 4 : 1;
  for (int i = threadIdx.x; i < kArrangeBytes / 16 * kBlocks * 32; i += blockDim.x) {
    const int l = i / 2 % 32, b = i / 64 % kBlocks;
    const int c = blockIdx.y * kArrangeBytes + (i % 2 + i / (64 * kBlocks) * 2) * 16;
    uint4 v[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int r = b * 128 + q * 32 + l;
      v[q] = make_uint4(0u, 0u, 0u, 0u);
      if (r < rows && c < sf_cols) v[q] = scale_words(src + static_cast<int64_t>(r) * stride, c, sf_cols, align);
    }
    // words c / 4 .. c / 4 + 3 of a row: K block, word in it
    const uint32_t* w[4] = {&v[0].x, &v[1].x, &v[2].x, &v[3].x};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int kb = c / (4 * kWords) + j / kWords;
      if (kb < num_kb)
        out[(static_cast<int64_t>(kb) * kBlocks * kWords + b * kWords + j % kWords) * 32 + l] =
            make_uint4(w[0][j], w[1][j], w[2][j], w[3][j]);
    }
  }
}

template <bool kNv, int kTokens, int kCols>
__global__ void __launch_bounds__(256) arrange_scales_kernel(const Fp4GemmArgs a) {
  constexpr int kWords = kNv ? 4 : 2;
  __shared__ int pre[kMaxExperts + 1], row_s[kMaxExperts + 1];
  wait_for_previous_kernel();
  int tile = blockIdx.x;
  if (tile < a.E * a.m_tiles) {
    const int g = tile / a.m_tiles, m = tile - g * a.m_tiles;
    // no row meets this expert (in whatever order the offsets are: rows of g are rows behind all before it)
    if (a.offsets && min(a.T, __ldg(a.offsets + g + 1)) <= max(0, __ldg(a.offsets + g))) return;
    const int rows = min(kCols, a.N - m * kCols);
    arrange_tile<kNv, kCols>(a.ws + (static_cast<int64_t>(g) * a.N + m * kCols) * a.ws_stride, a.ws_stride, rows,
                             a.sf_cols, a.num_kb,
                             reinterpret_cast<uint4*>(a.ws_tiles) +
                                 static_cast<int64_t>(tile) * a.num_kb * ((kCols + 127) / 128 * kWords * 32));
    return;
  }
  tile -= a.E * a.m_tiles;
  if (threadIdx.x < 32) scan_experts<kTokens>(a.offsets, a.E, a.T, pre, row_s);
  __syncthreads();
  if (tile >= pre[a.E]) return;
  int lo = 0, hi = a.E - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (pre[mid] <= tile) lo = mid; else hi = mid - 1;
  }
  const int row0 = row_s[lo] + (tile - pre[lo]) * kTokens;
  arrange_tile<kNv, kTokens>(a.xs + static_cast<int64_t>(row0) * a.xs_stride, a.xs_stride,
                             min(kTokens, row_s[lo + 1] - row0), a.sf_cols, a.num_kb,
                             reinterpret_cast<uint4*>(a.xs_tiles) +
                                 static_cast<int64_t>(tile) * a.num_kb * ((kTokens + 127) / 128 * kWords * 32));
}

template <bool kNv, int kTokens, int kCols>
cudaError_t launch_arrange(const Fp4GemmArgs& a, int64_t xtiles, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>(static_cast<int64_t>(a.E) * a.m_tiles + xtiles), (a.num_kb * (kNv ? 16 : 8) + kArrangeBytes - 1) / kArrangeBytes);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, arrange_scales_kernel<kNv, kTokens, kCols>, a);
}

template <bool kNv>
cudaError_t launch_fmt(const CUtensorMap& tw, const CUtensorMap& tx, const Fp4GemmArgs& a, const Fp4Plan& p,
                       int num_sms, cudaStream_t s) {
  const int64_t xtiles = a.E == 1 ? (a.T + p.tokens - 1) / p.tokens : a.T / p.tokens + (a.E < a.T ? a.E : a.T);
  const int64_t most = xtiles * a.m_tiles;
  if (p.tokens > 32) {
    const cudaError_t e = p.tokens == 192 ? launch_arrange<kNv, 192, 256>(a, xtiles, s)
                          : p.cols == 256 ? launch_arrange<kNv, 96, 256>(a, xtiles, s)
                                          : launch_arrange<kNv, 96, 128>(a, xtiles, s);
    if (e != cudaSuccess) return e;
  }
  if (p.splits > 1) return launch_cfg<kNv, false, 1, 32, true>(tw, tx, a, static_cast<int>(most) * p.splits, s);
  const int grid = static_cast<int>(most < num_sms ? most : num_sms);
  if (p.tokens == 32)
    return p.cols == 128 ? launch_cfg<kNv, false, 1, 32, false>(tw, tx, a, grid, s)
                         : launch_cfg<kNv, false, 2, 32, false>(tw, tx, a, grid, s);
  if (p.cols == 128) return launch_cfg<kNv, true, 1, 96, false>(tw, tx, a, grid, s);
  if (p.tokens == 96) return launch_cfg<kNv, true, 2, 96, false>(tw, tx, a, grid, s);
  return launch_cfg<kNv, true, 2, 192, false>(tw, tx, a, grid, s);
}

}  // namespace

// Bytes of one tile's arranged scales of one K block.
static int64_t tile_sf_bytes(int format, int rows) { return (rows + 127) / 128 * (format == kFp4Nv ? 4 : 2) * 512; }
static int64_t token_tiles(int T, int E, int tokens) {
  // at most T / tokens whole ones, and one partial one for each expert that has rows
  return E == 1 ? (T + tokens - 1) / tokens : T / tokens + (E < T ? E : T);
}

int64_t fp4_workspace(int format, int T, int N, int E, int num_kb, const Fp4Plan& p) {
  if (p.tokens == 32) return 0;
  const int64_t wt = static_cast<int64_t>(E) * ((N + p.cols - 1) / p.cols);
  return num_kb * (wt * tile_sf_bytes(format, p.cols) + token_tiles(T, E, p.tokens) * tile_sf_bytes(format, p.tokens));
}

static int max_clusters(int size) {
  // per device and size, asked once: what a device can hold does not change
  constexpr int kDevices = 64;
  static std::atomic<int> known[kDevices][kMaxSplits + 1];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kDevices) return 0;
  const int have = known[dev][size].load(std::memory_order_relaxed);
  if (have > 0) return have - 1;
  using C = Cfg<true, false, 1, 32>;
  auto* kernel = gemm_fp4_kernel<true, false, 1, 32, true>;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(size);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::kSmemBytes;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = size;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes) != cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
    cudaGetLastError();
    return 0;  // not kept: the next call asks again
  }
  known[dev][size].store(n + 1, std::memory_order_relaxed);
  return n;
}

// Largest number of CTAs per cluster with which `tiles` clusters are on the device at once and each has a K
// block. A cluster's CTAs sit in one GPC, whose SMs are no multiple of every size: a second round of clusters
// costs more than it brings (36 tiles: 14.7 us with 4 CTAs each, of which 33 clusters fit, 8.2 us with 3).
static int splits_for(int64_t tiles, int num_kb) {
  for (int s = kMaxSplits; s > 1; --s)
    if (s <= num_kb && tiles <= max_clusters(s)) return s;
  return 1;
}

// Tile shape. Up to 32 rows per expert (on average, where there are several) a tile is 32 tokens wide; its
// height is 256 rows of w where that still gives every SM a tile, else 128, and where even those leave SMs
// idle a cluster shares each tile's K. With more rows, the shape whose rounds of tiles cost least; several
// experts' weights, which HBM bounds, are read in wide token tiles only.
Fp4Plan fp4_plan(int T, int N, int E, int num_kb, int num_sms) {
  // ns of each shape: once (launches, the arrangement of the scales, the first stages), per tile (epilogue),
  // per stage; fitted to eleven shapes from 48 x 4608 x 5120 to 4096 x 1024 x 1024, which they meet to 15 %
  constexpr struct {
    int tokens, cols, once, tile, stage;
  } kShapes[] = {{192, 256, 6000, 5000, 560},
                 {96, 256, 6000, 2700, 455},
                 {96, 128, 6000, 2500, 325},
                 {32, 256, 4700, 300, 530},
                 {32, 128, 4100, 1600, 290}};
  constexpr int kJoin = 1300;  // a split tile's sum
  const int per = (T + E - 1) / E, experts = E < T ? E : T;
  Fp4Plan p{32, 256, 1};
  int64_t least = INT64_MAX;
  for (const auto& sh : kShapes) {
    if (per <= 32 ? sh.tokens > 32 : E > 1 && sh.tokens == 32) continue;
    // one matrix: its tiles; several: an expert's last tile is half full on average
    const int64_t tok = E == 1      ? (T + sh.tokens - 1) / sh.tokens
                        : per <= 32 ? experts
                                    : T / sh.tokens + (E + 1) / 2;
    const int64_t tiles = tok * ((N + sh.cols - 1) / sh.cols);
    int splits = 1;
    if (sh.tokens == 32 && sh.cols == 128) splits = splits_for(tiles, num_kb);
    const int64_t rounds = (tiles + num_sms - 1) / num_sms, stages = (num_kb + splits - 1) / splits;
    const int64_t cost = sh.once + rounds * (sh.tile + stages * sh.stage) + (splits > 1 ? kJoin : 0);
    if (cost < least) {
      least = cost;
      p = Fp4Plan{sh.tokens, sh.cols, splits};
    }
  }
  return p;
}

cudaError_t take_fp4_status(int* v) {
  cudaError_t e = cudaDeviceSynchronize();
  if (e == cudaSuccess) e = cudaMemcpyFromSymbol(v, product_status, sizeof(int));
  const int zero = 0;
  if (e == cudaSuccess && *v != 0) e = cudaMemcpyToSymbol(product_status, &zero, sizeof(int));
  return e;
}

cudaError_t launch_gemm_fp4(int format, const CUtensorMap& tw, const CUtensorMap& tx, Fp4GemmArgs a, void* workspace,
                            const Fp4Plan& p, int num_sms, cudaStream_t s) {
  if (a.E > kMaxExperts) return cudaErrorInvalidValue;
  a.ws_tiles = static_cast<uint8_t*>(workspace);
  a.xs_tiles = a.ws_tiles + static_cast<int64_t>(a.num_kb) * a.E * a.m_tiles * tile_sf_bytes(format, p.cols);
  return format == kFp4Nv ? launch_fmt<true>(tw, tx, a, p, num_sms, s) : launch_fmt<false>(tw, tx, a, p, num_sms, s);
}

}  // namespace moe
