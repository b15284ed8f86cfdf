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
//   warp 0      TMA: w box 256 values (128 bytes) x 128 kHalves rows, x boxes x 32 rows
//   warp 1      issues the MMAs, four K = 64 steps per ring stage
//   warps 2-5   scale factors, one warp per TMEM lane quarter: shared memory -> registers ->
//               TMEM with tcgen05.st. The MMA wants every row's scales in lane row % 32,
//               column row / 32, replicated in the four quarters, which is how the four
//               warps write them, so the scales stay in rows of K / 32 or K / 16 bytes in
//               HBM and are rearranged nowhere
//   warps 6-13  epilogue, two per lane quarter taking interleaved 16-column chunks
//   warp 14     copies the scale rows of a stage into a ring of their own (cp.async, 16 or 8
//               bytes a row, zeros where a row or its end is outside), several stages ahead:
//               loaded by the warps that store them, one stage ahead, a load's latency set
//               the time of a stage (T 8192, N 4608, K 5120: 650 us against 207 with this ring)
//
// Few tokens and few tiles: a cluster of `splits` CTAs takes one tile, each a slice of K;
// the partial tiles meet in the first CTA's shared memory and are summed in slice order.
//
// Every read of offsets is clamped to [0, T] and to ascending order, so no offsets lead
// outside x or y. All waits are bounded.
#include <cuda_fp16.h>

#include "common.cuh"
#include "kernels.h"

namespace moe {

namespace {

constexpr int kSfWarps = 4;
constexpr int kEpiWarps = 8;
constexpr int kEpiGroups = kEpiWarps / 4;
constexpr int kFirstSf = 2;
constexpr int kFirstEpi = kFirstSf + kSfWarps;
constexpr int kSfLoader = kFirstEpi + kEpiWarps;
constexpr int kThreads = 32 * (kSfLoader + 1);
constexpr int kBK = 256;              // K values per stage
constexpr int kRowBytes = kBK / 2;    // 128: one swizzle row
constexpr int kBox = 32;              // token rows per TMA box
constexpr int kMaxExperts = 512;
constexpr int kMaxSplits = 8;

// kHalves: 128-row halves of w per tile; kBN: token rows per tile.
template <bool kNv, int kHalves, int kBN>
struct Cfg {
  static constexpr int kABytes = kHalves * 128 * kRowBytes;
  static constexpr int kBBytes = kBN * kRowBytes;
  static constexpr int kAtoms = kNv ? 4 : 2;                       // 32-bit words of scales per row and stage
  static constexpr int kBCols = (kBN / 32 + 3) / 4 * 4;            // TMEM columns of one atom of x's scales
  static constexpr int kSfCols = kAtoms * (4 * kHalves + kBCols);  // ... of one stage's scales
  static constexpr int kAccCols = kHalves * kBN;
  static constexpr int kAccs = 2 * kAccCols + 2 * kSfCols <= 512 ? 2 : 1;
  static constexpr int kSets = (512 - kAccs * kAccCols) / kSfCols >= 4 ? 4 : (512 - kAccs * kAccCols) / kSfCols;
  static constexpr int kSfBase = kAccs * kAccCols;
  static constexpr int kFixed = 1024 + 512 + 2 * (kMaxExperts + 1) * 4;  // alignment, barriers, experts
  static constexpr int kRowSf = kNv ? 16 : 8;                      // scale bytes of a row and stage
  static constexpr int kRawBytes = (128 * kHalves + kBN) * kRowSf;
  static constexpr int kRaw = 6;                                   // stages of scales in flight
  static constexpr int kFit = (227 * 1024 - kFixed - kRaw * kRawBytes) / (kABytes + kBBytes);
  static constexpr int kStages = kFit > 8 ? 8 : kFit;
  static constexpr int kSmemBytes = kFixed + kRaw * kRawBytes + kStages * (kABytes + kBBytes);
  static_assert(kSets >= 2, "scale factors of two stages");
  static_assert((2 * kStages + 2 * kSets + 2 * kAccs + 2 * kRaw + 1) * 8 + 8 <= 512, "barriers");
  // the partial tiles of a split fit in the ring (kHalves == 1, kBN == 32)
  static_assert(kHalves > 1 || kBN > 32 || (kMaxSplits - 1) * 128 * 32 * 4 <= kStages * (kABytes + kBBytes), "split");
};

// Instruction descriptor of the 4-bit kinds: E2M1 is format 1 (A bits 7-9, B bits 10-12), both
// K-major, N >> 3 in bits 17-22, scale format in bit 23 (1: E8M0, 0: E4M3), M >> 4 in bits 24-28,
// scale-factor ids in bits 4-5 (B) and 29-30 (A), K = 64 (bit 31 = 0).
__device__ __forceinline__ uint32_t idesc_fp4(bool nv, uint32_t N, uint32_t sf_id) {
  return (sf_id << 4) | (1u << 7) | (1u << 10) | ((N >> 3) << 17) | ((nv ? 0u : 1u) << 23) | ((128u >> 4) << 24) |
         (sf_id << 29);
}

template <bool kNv>
__device__ __forceinline__ void umma_fp4(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t sfa,
                                         uint32_t sfb, uint32_t accumulate) {
  if constexpr (kNv)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%5], [%6], p;\n\t}\n" ::
            "r"(d),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%5], [%6], p;\n\t}\n" ::"r"(
            d),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb)
        : "memory");
}

// Four consecutive 32-bit TMEM columns of this warp's lane quarter.
__device__ __forceinline__ void tmem_st4(uint32_t taddr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr), "r"(a), "r"(b), "r"(c),
               "r"(d)
               : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ uint32_t cluster_ctarank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Store to the same shared-memory address of another CTA of the cluster.
__device__ __forceinline__ void st_cluster_f32(uint32_t saddr, uint32_t rank, float v) {
  asm volatile(
      "{\n\t.reg .b32 a;\n\t"
      "mapa.shared::cluster.u32 a, %0, %1;\n\t"
      "st.shared::cluster.f32 [a], %2;\n\t}\n" ::"r"(saddr),
      "r"(rank), "f"(v)
      : "memory");
}

__device__ __forceinline__ bool wait_or_abort(uint64_t* bar, uint32_t parity, const Fp4GemmArgs& a,
                                              volatile int* abort_flag) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 32; ++i)
      if (mbar_try_wait(bar, parity)) return true;
    if (*abort_flag) return false;
    if (globaltimer_ns() - t0 > a.timeout_ns) {
      *abort_flag = 1;
      report_status(a.status, kStatusTimeout);
      return false;
    }
  }
}

struct Tile {
  int g, m, row0, nrows;
};

// Tile t: experts in order, inside an expert the w tiles in order, inside a w tile its token
// tiles, so that CTAs taking consecutive tiles read the same weights together, through L2.
// `pre` holds each expert's first token tile, `row` its first row.
template <int kBN>
__device__ __forceinline__ Tile tile_of(int t, int E, int m_tiles, const int* pre, const int* row) {
  int lo = 0, hi = E - 1;
  const int want = t / m_tiles;  // pre[g] * m_tiles <= t  <=>  pre[g] <= t / m_tiles
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (pre[mid] <= want) lo = mid; else hi = mid - 1;
  }
  const int nt = pre[lo + 1] - pre[lo];
  const int local = t - pre[lo] * m_tiles;
  Tile r;
  r.g = lo;
  r.m = local / nt;
  const int n = local % nt;
  r.row0 = row[lo] + n * kBN;
  r.nrows = min(kBN, row[lo + 1] - r.row0);
  return r;
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

template <typename T>
__device__ __forceinline__ T round_out(float v);
template <>
__device__ __forceinline__ float round_out<float>(float v) {
  return v;
}
template <>
__device__ __forceinline__ __nv_bfloat16 round_out<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}
template <>
__device__ __forceinline__ __half round_out<__half>(float v) {
  return __float2half_rn(v);
}

// 16 columns (tokens) of one output row n = m of w: lanes hold consecutive n.
template <typename T>
__device__ __forceinline__ void store_chunk(void* out, int64_t ld, int row0, int c0, int nrows, int n, bool n_ok,
                                            float alpha, const uint32_t (&r)[16]) {
  if (!n_ok) return;
  T* p = static_cast<T*>(out) + static_cast<int64_t>(row0 + c0) * ld + n;
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    if (c0 + j < nrows) *p = round_out<T>(alpha * __uint_as_float(r[j]));
    p += ld;
  }
}
__device__ __forceinline__ void store_any(const Fp4GemmArgs& a, int row0, int c0, int nrows, int n, bool n_ok,
                                          float alpha, const uint32_t (&r)[16]) {
  if (a.out_dtype == kValBf16)
    store_chunk<__nv_bfloat16>(a.out, a.N, row0, c0, nrows, n, n_ok, alpha, r);
  else if (a.out_dtype == kValFp16)
    store_chunk<__half>(a.out, a.N, row0, c0, nrows, n, n_ok, alpha, r);
  else
    store_chunk<float>(a.out, a.N, row0, c0, nrows, n, n_ok, alpha, r);
}

template <bool kNv, int kHalves, int kBN, bool kSplit>
__global__ void __launch_bounds__(kThreads, 1)
    gemm_fp4_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                    const Fp4GemmArgs args) {
  using C = Cfg<kNv, kHalves, kBN>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sA = smem;
  uint8_t* sB = sA + C::kStages * C::kABytes;
  uint8_t* sRaw = sB + C::kStages * C::kBBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sRaw + C::kRaw * C::kRawBytes);
  uint64_t* full = bars;
  uint64_t* empty = full + C::kStages;
  uint64_t* sffull = empty + C::kStages;
  uint64_t* sfempty = sffull + C::kSets;
  uint64_t* tfull = sfempty + C::kSets;
  uint64_t* tempty = tfull + C::kAccs;
  uint64_t* rfull = tempty + C::kAccs;
  uint64_t* rempty = rfull + C::kRaw;
  uint64_t* drain = rempty + C::kRaw;
  uint32_t* tmem_base_smem = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_base_smem + 1);
  int* pre = reinterpret_cast<int*>(reinterpret_cast<uint8_t*>(bars) + 512);  // [E + 1] first token tile
  int* row_s = pre + kMaxExperts + 1;                                         // [E + 1] first row

  const int warp = threadIdx.x / 32;
  const int lane = threadIdx.x % 32;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < C::kSets; ++i) {
      mbar_init(&sffull[i], kSfWarps);
      mbar_init(&sfempty[i], 1);
    }
    for (int i = 0; i < C::kAccs; ++i) {
      mbar_init(&tfull[i], 1);
      mbar_init(&tempty[i], kEpiWarps);
    }
    for (int i = 0; i < C::kRaw; ++i) {
      mbar_init(&rfull[i], 32);
      mbar_init(&rempty[i], kSfWarps);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbarrier_init();
    tma_prefetch_desc(&tmW);
    tma_prefetch_desc(&tmX);
  }
  if (warp == 1) {
    tmem_alloc(tmem_base_smem, 512);
    tmem_relinquish();
  }
  // the experts' rows and token tiles: warp 2 scans 32 experts at a time
  if (warp == kFirstSf) {
    int last = 0, tiles = 0;
    for (int b = 0; b <= args.E; b += 32) {
      const int g = b + lane;
      int v = 0;
      if (g <= args.E) v = args.offsets ? max(0, min(args.T, __ldg(args.offsets + g))) : (g == 0 ? 0 : args.T);
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
      int n = g > 0 && g <= args.E ? (v - before + kBN - 1) / kBN : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, n, o);
        if (lane >= o) n += u;
      }
      if (g <= args.E) {
        row_s[g] = v;
        pre[g] = tiles + n;
      }
      tiles += __shfl_sync(0xffffffffu, n, 31);
      last = __shfl_sync(0xffffffffu, v, 31);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_base_smem;
  const int total = pre[args.E] * args.m_tiles;

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
        const Tile tl = tile_of<kBN>(t, args.E, args.m_tiles, pre, row_s);
        const int w_row = tl.g * args.N + tl.m * 128 * kHalves;
        const int nb = (tl.nrows + kBox - 1) / kBox;
        bool ok = true;
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!wait_or_abort(&empty[stage], phase ^ 1, args, abort_flag)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&full[stage], C::kABytes + nb * kBox * kRowBytes);
          tma_load_2d(sA + stage * C::kABytes, &tmW, &full[stage], kb * kRowBytes, w_row, kCacheEvictFirst);
          for (int j = 0; j < nb; ++j)
            tma_load_2d(sB + stage * C::kBBytes + j * kBox * kRowBytes, &tmX, &full[stage], kb * kRowBytes,
                        tl.row0 + j * kBox, kCacheEvictLast);
          ++issued;
          if (++stage == C::kStages) {
            stage = 0;
            phase ^= 1;
          }
        }
        if (!ok) break;
      }
      if (*abort_flag) {
        // let the copies in flight land before the CTA's shared memory goes
        for (long i = issued - 1; i >= 0 && i >= issued - C::kStages; --i) {
          const uint64_t b = globaltimer_ns();
          while (!mbar_try_wait(&full[i % C::kStages], static_cast<uint32_t>((i / C::kStages) & 1)) &&
                 globaltimer_ns() - b < args.timeout_ns) {
          }
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      int stage = 0, set = 0, acc = 0;
      uint32_t phase = 0, sphase = 0, aphase = 0;
      for (int t = t0; t < total && !*abort_flag; t += stride) {
        const Tile tl = tile_of<kBN>(t, args.E, args.m_tiles, pre, row_s);
        const uint32_t n_mma = (tl.nrows + 15) & ~15;
        if (!wait_or_abort(&tempty[acc], aphase ^ 1, args, abort_flag)) break;
        tc_fence_after();
        const uint32_t d = tmem_base + acc * C::kAccCols;
        bool ok = true;
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!wait_or_abort(&full[stage], phase, args, abort_flag) ||
              !wait_or_abort(&sffull[set], sphase, args, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t a_addr = smem_u32(sA + stage * C::kABytes);
          const uint32_t b_addr = smem_u32(sB + stage * C::kBBytes);
          const uint32_t sf = tmem_base + C::kSfBase + set * C::kSfCols;
#pragma unroll
          for (uint32_t j = 0; j < 4; ++j) {
            const uint32_t atom = kNv ? j : j / 2, id = kNv ? 0 : (j & 1) * 2;
            const uint32_t idesc = idesc_fp4(kNv, n_mma, id);
            const uint64_t bdesc = sdesc_sw128(b_addr + j * 32);
            const uint32_t sfb = (sf + kHalves * C::kAtoms * 4 + atom * C::kBCols) | (id << 30);
#pragma unroll
            for (uint32_t h = 0; h < kHalves; ++h)
              umma_fp4<kNv>(d + h * kBN, sdesc_sw128(a_addr + h * 128 * kRowBytes + j * 32), bdesc, idesc,
                            (sf + (h * C::kAtoms + atom) * 4) | (id << 30), sfb, kb != kb0 || j != 0);
          }
          umma_commit(&empty[stage]);
          umma_commit(&sfempty[set]);
          if (++stage == C::kStages) {
            stage = 0;
            phase ^= 1;
          }
          if (++set == C::kSets) {
            set = 0;
            sphase ^= 1;
          }
        }
        if (!ok) break;
        umma_commit(&tfull[acc]);
        if (++acc == C::kAccs) {
          acc = 0;
          aphase ^= 1;
        }
      }
      // every MMA done before TMEM and shared memory go
      umma_commit(drain);
      const uint64_t b = globaltimer_ns();
      while (!mbar_try_wait(drain, 0) && globaltimer_ns() - b < args.timeout_ns) {
      }
    }
  } else if (warp < kFirstEpi) {
    // ------------------------------------------------------------ scale factors -> TMEM
    constexpr int kW = C::kAtoms;
    constexpr int kARows = 4 * kHalves, kBRows = kBN / 32;  // rows of this lane: 32 apart
    const uint32_t quarter = tmem_base + (static_cast<uint32_t>((warp & 3) * 32) << 16) + C::kSfBase;
    int set = 0, raw = 0;
    uint32_t sphase = 0, rphase = 0;
    bool ok = true;
    for (int t = t0; ok && t < total; t += stride) {
      for (int kb = kb0; kb < kb1; ++kb) {
        if (lane == 0)
          ok = wait_or_abort(&rfull[raw], rphase, args, abort_flag) &&
               wait_or_abort(&sfempty[set], sphase ^ 1, args, abort_flag);
        ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
        if (!ok) break;
        tc_fence_after();
        const uint8_t* src = sRaw + raw * C::kRawBytes + lane * C::kRowSf;
        const uint32_t base = quarter + set * C::kSfCols;
#pragma unroll
        for (int h = 0; h < kHalves; ++h) {
          uint32_t w[4 * kW];
#pragma unroll
          for (int i = 0; i < 4; ++i) read_scales<kW>(src + (4 * h + i) * 32 * C::kRowSf, w + i * kW);
#pragma unroll
          for (int j = 0; j < kW; ++j) tmem_st4(base + (h * kW + j) * 4, w[j], w[kW + j], w[2 * kW + j], w[3 * kW + j]);
        }
#pragma unroll
        for (int c = 0; c < C::kBCols; c += 4) {
          uint32_t w[4 * kW];
#pragma unroll
          for (int i = 0; i < 4 * kW; ++i) w[i] = 0u;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (c + i < kBRows) read_scales<kW>(src + (kARows + c + i) * 32 * C::kRowSf, w + i * kW);
#pragma unroll
          for (int j = 0; j < kW; ++j)
            tmem_st4(base + kHalves * kW * 4 + j * C::kBCols + c, w[j], w[kW + j], w[2 * kW + j], w[3 * kW + j]);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&rempty[raw]);
          mbar_arrive(&sffull[set]);
        }
        if (++set == C::kSets) {
          set = 0;
          sphase ^= 1;
        }
        if (++raw == C::kRaw) {
          raw = 0;
          rphase ^= 1;
        }
      }
    }
  } else if (warp == kSfLoader) {
    // ------------------------------------------------------------ scale rows -> shared memory
    constexpr int kB = C::kRowSf;
    int raw = 0;
    uint32_t rphase = 0;
    bool ok = true;
    for (int t = t0; ok && t < total; t += stride) {
      const Tile tl = tile_of<kBN>(t, args.E, args.m_tiles, pre, row_s);
      const int n = tl.m * 128 * kHalves + lane;
      const int w_left = args.N - n, x_left = tl.nrows - lane;  // rows from this lane's first one
      const uint8_t* wrow = args.ws + (static_cast<int64_t>(tl.g) * args.N + n) * args.ws_stride;
      const uint8_t* xrow = args.xs + static_cast<int64_t>(tl.row0 + lane) * args.xs_stride;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (lane == 0) ok = wait_or_abort(&rempty[raw], rphase ^ 1, args, abort_flag);
        ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
        if (!ok) break;
        const uint32_t dst = smem_u32(sRaw + raw * C::kRawBytes + lane * kB);
        const int off = kb * kB;
        const int left = min(kB, args.sf_cols - off);
        // a row outside reads nothing (0 bytes from the scales' own start)
#pragma unroll
        for (int i = 0; i < 4 * kHalves; ++i) {
          const bool in = 32 * i < w_left;
          cp_async_zfill<kB>(dst + i * 32 * kB, in ? wrow + static_cast<int64_t>(i) * 32 * args.ws_stride + off : args.ws,
                             in ? left : 0);
        }
#pragma unroll
        for (int i = 0; i < kBN / 32; ++i) {
          const bool in = 32 * i < x_left;
          cp_async_zfill<kB>(dst + (4 * kHalves + i) * 32 * kB,
                             in ? xrow + static_cast<int64_t>(i) * 32 * args.xs_stride + off : args.xs, in ? left : 0);
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
  } else {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3;
    const int cfirst = ((warp - kFirstEpi) / 4) * 16;
    const float xts = args.x_ts ? __ldg(args.x_ts) : 1.0f;
    int acc = 0;
    uint32_t aphase = 0;
    for (int t = t0; t < total; t += stride) {
      const Tile tl = tile_of<kBN>(t, args.E, args.m_tiles, pre, row_s);
      bool ok = true;
      if (lane == 0) ok = wait_or_abort(&tfull[acc], aphase, args, abort_flag);
      ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
      if (!ok) break;
      tc_fence_after();
      if constexpr (!kSplit) {
        const float alpha = args.w_ts ? xts * __ldg(args.w_ts + tl.g) : xts;
        const uint32_t tb = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + acc * C::kAccCols;
        const int n = tl.m * 128 * kHalves + q * 32 + lane;
        for (int c0 = cfirst; c0 < tl.nrows; c0 += 16 * kEpiGroups) {
#pragma unroll
          for (int h = 0; h < kHalves; ++h) {
            uint32_t r[16];
            tmem_ld16(tb + h * kBN + c0, r);
            tmem_ld_wait();
            store_any(args, tl.row0, c0, tl.nrows, n + h * 128, n + h * 128 < args.N, alpha, r);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&tempty[acc]);
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
    const int cfirst = ((warp - kFirstEpi) / 4) * 16;
    const bool work = warp >= kFirstEpi && warp < kSfLoader && t0 < total && !*abort_flag;
    Tile tl{};
    if (work) tl = tile_of<kBN>(t0, args.E, args.m_tiles, pre, row_s);
    uint32_t r[16];
    if (work && cfirst < tl.nrows) {
      tc_fence_after();
      tmem_ld16(tmem_base + (static_cast<uint32_t>(q * 32) << 16) + cfirst, r);
      tmem_ld_wait();
      if (rank != 0) {
        const uint32_t dst = smem_u32(sA) + (((rank - 1) * kBN + cfirst) * 128 + q * 32 + lane) * 4;
#pragma unroll
        for (int j = 0; j < 16; ++j) st_cluster_f32(dst + j * 512, 0, __uint_as_float(r[j]));
      }
    }
    __syncwarp();
    cluster_sync_all();
    if (work && rank == 0 && cfirst < tl.nrows) {
      const float* part = reinterpret_cast<const float*>(sA) + cfirst * 128 + q * 32 + lane;
      for (int p = 0; p < splits - 1; ++p)
#pragma unroll
        for (int j = 0; j < 16; ++j)
          r[j] = __float_as_uint(__uint_as_float(r[j]) + part[(p * kBN + j) * 128]);
      const float xts = args.x_ts ? __ldg(args.x_ts) : 1.0f;
      const float alpha = args.w_ts ? xts * __ldg(args.w_ts + tl.g) : xts;
      const int n = tl.m * 128 + q * 32 + lane;
      store_any(args, tl.row0, cfirst, tl.nrows, n, n < args.N, alpha, r);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, 512);
  }
}

template <bool kNv, int kHalves, int kBN, bool kSplit>
cudaError_t launch_cfg(const CUtensorMap& tw, const CUtensorMap& tx, const Fp4GemmArgs& a, int grid, cudaStream_t s) {
  using C = Cfg<kNv, kHalves, kBN>;
  auto* kernel = gemm_fp4_kernel<kNv, kHalves, kBN, kSplit>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::kSmemBytes;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = kSplit ? a.splits : 1;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = kSplit ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, tw, tx, a);
}

template <bool kNv>
cudaError_t launch_fmt(const CUtensorMap& tw, const CUtensorMap& tx, const Fp4GemmArgs& a, const Fp4Plan& p,
                       int num_sms, cudaStream_t s) {
  // token tiles: at most T / bn whole ones, and one partial one for each expert that has rows
  const int64_t tok = a.E == 1 ? (a.T + p.bn - 1) / p.bn : a.T / p.bn + (a.E < a.T ? a.E : a.T);
  const int64_t most = tok * a.m_tiles;
  if (p.splits > 1)
    return launch_cfg<kNv, 1, 32, true>(tw, tx, a, static_cast<int>(most) * p.splits, s);
  const int grid = static_cast<int>(most < num_sms ? most : num_sms);
  if (p.halves == 1) return launch_cfg<kNv, 1, 32, false>(tw, tx, a, grid, s);
  if (p.bn == 32) return launch_cfg<kNv, 2, 32, false>(tw, tx, a, grid, s);
  if (p.bn == 96) return launch_cfg<kNv, 2, 96, false>(tw, tx, a, grid, s);
  return launch_cfg<kNv, 2, 192, false>(tw, tx, a, grid, s);
}

}  // namespace

// Tile shape. Up to 32 rows per expert (on average, where there are several) a tile is 32 tokens
// wide; its height is 256 rows of w where that still gives every SM a tile, else 128, and
// where even those leave SMs idle a cluster shares each tile's K.
Fp4Plan fp4_plan(int T, int N, int E, int num_kb, int num_sms) {
  Fp4Plan p{2, 32, 1};
  const int per = (T + E - 1) / E;
  if (per > 96) {
    p.bn = 192;
    return p;
  }
  if (per > 32) {
    p.bn = 96;
    return p;
  }
  const int experts = E < T ? E : T;
  if (static_cast<int64_t>(experts) * ((N + 255) / 256) >= num_sms) return p;
  p.halves = 1;
  const int tiles = experts * ((N + 127) / 128);
  while (p.splits < kMaxSplits && tiles * p.splits * 2 <= num_sms && p.splits * 2 <= num_kb) p.splits *= 2;
  return p;
}

cudaError_t launch_gemm_fp4(int format, const CUtensorMap& tw, const CUtensorMap& tx, const Fp4GemmArgs& a,
                            const Fp4Plan& p, int num_sms, cudaStream_t s) {
  if (a.E > kMaxExperts) return cudaErrorInvalidValue;
  return format == kFp4Nv ? launch_fmt<true>(tw, tx, a, p, num_sms, s) : launch_fmt<false>(tw, tx, a, p, num_sms, s);
}

}  // namespace moe
