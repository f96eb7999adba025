// W8A8 matrix product with one scale per token and one per output channel
// (sm_100a tensor cores).
//
// Quamba2 (shd-paper.top card), abstract: W8A8, 8-bit weights times 8-bit
// activations.  y[t][n] = round(acc (x_scale[t] w_scale[n]) + bias[n]) with
// acc = sum_k x[t][k] w[n][k] in 32-bit integers (tcgen05.mma kind::i8), so
// the sum is exact and its order does not matter.
//
// Orientation: the weights are the MMA's A operand (its M rows are output
// channels) and the tokens its B operand (its N columns), at every size.  An
// accumulator lane is then a channel and a column a token, so N follows the
// token count down to 16 without idle MMA rows, and the 32 lanes of a warp
// store 32 consecutive channels of one token: whole sectors straight from
// registers, at any alignment.
//
// Both operands are K-major, brought in by TMA as 128-byte rows in the
// 128-byte swizzle (32 bytes, one MMA K-step, per quarter row); rows and
// columns beyond the tensor read as zero.
#include "internal.h"
#include "stream.cuh"
#include "tc.cuh"
#include "tma_map.h"
#include "vec8.cuh"

namespace ssmq {
namespace {

constexpr int kBlockK = 128;                 // bytes of K per stage
constexpr int kRows = 128;                   // operand rows of one TMA box (weights)
constexpr int kOperand = kRows * kBlockK;    // 16 KB
constexpr uint32_t kWaitLimit = 1u << 20;

struct LinParams {
  int64_t M, N;      // tokens, channels
  int kblocks;
  const float* xs;
  const float* ws;
  const float* bias;
  void* y;
  int64_t ldy;
  int dtype;
  uint32_t* status;
  int64_t tok_tiles, ch_tiles, group;  // persistent kernel: tile order
  bool tma_out;                        // and whether y goes out by TMA
  // probes before a wait of the copies' or the epilogue's threads gives up (the MMA
  // thread's waits keep kWaitLimit: with a limit from memory its loop is slower, 145.5
  // against 140.5 us at 16384 x 2560 x 5120)
  uint32_t wait_limit;
};

// ---- PTX ---------------------------------------------------------------------
__device__ __forceinline__ uint32_t mapa(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ uint32_t cta_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* map, int k, int row,
                                         uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], "
      "[%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(map), "r"(k), "r"(row), "r"(bar)
      : "memory");
}
// the same for a CTA pair: bar may lie in either CTA of the pair
__device__ __forceinline__ void tma_load_pair(uint32_t dst, const CUtensorMap* map, int k, int row,
                                              uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".cta_group::2 [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(map), "r"(k), "r"(row), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}
// K-major operand in the 128-byte swizzle: 8-row groups 1024 bytes apart
__device__ __forceinline__ uint64_t sw128_desc(uint32_t saddr) {
  uint64_t d = (uint64_t)((saddr >> 4) & 0x3FFFu);
  d |= (uint64_t)1u << 16;
  d |= (uint64_t)(1024u >> 4) << 32;
  d |= (uint64_t)1u << 46;
  d |= (uint64_t)2u << 61;
  return d;
}
// kind::i8: signed A and B, 32-bit integer accumulator
__host__ __device__ constexpr uint32_t idesc_i8(int M, int N) {
  return (2u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) |
         ((uint32_t)(M >> 4) << 24);
}
template <int kGroup>
__device__ __forceinline__ void mma_i8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       uint32_t accumulate) {
  if constexpr (kGroup == 1)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate));
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate));
}
// arrive on `bar` of both CTAs of the pair once this thread's MMAs are done
__device__ __forceinline__ void commit_pair(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
      "[%0], %1;" ::"r"(tc::smem_u32(bar)),
      "h"((uint16_t)3)
      : "memory");
}
// what a barrier of this CTA still expects, less `bytes` that will not come
__device__ __forceinline__ void complete_tx(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.complete_tx.relaxed.cluster.shared::cluster.b64 [%0], %1;" ::"r"(
                   tc::smem_u32(bar)),
               "r"(bytes)
               : "memory");
}
// a word of another CTA's shared memory (an address from mapa)
__device__ __forceinline__ void store_remote(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void store_remote64(uint32_t addr, int64_t v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}
// whether `ok` holds in all `n` threads that meet at named barrier `id`
__device__ __forceinline__ bool all_of(uint32_t id, uint32_t n, bool ok) {
  uint32_t r;
  __syncwarp();
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %3, 0;\n\t"
      "bar.red.and.pred q, %1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}\n"
      : "=r"(r)
      : "r"(id), "r"(n), "r"((uint32_t)ok)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void arrive_remote(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar)
               : "memory");
}
// 32 (16) columns of this thread's TMEM lane; usable after tmem_done, through
// which the registers pass so that no use moves in front of the wait
__device__ __forceinline__ void tmem_get(uint32_t taddr, int (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, "
      "%30, %31}, [%32];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
        "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]),
        "=r"(v[14]), "=r"(v[15]), "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]),
        "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]), "=r"(v[25]),
        "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_get(uint32_t taddr, int (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15}, [%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
        "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]),
        "=r"(v[14]), "=r"(v[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_done(int (&v)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]),
                 "+r"(v[6]), "+r"(v[7]), "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]),
                 "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15]), "+r"(v[16]), "+r"(v[17]),
                 "+r"(v[18]), "+r"(v[19]), "+r"(v[20]), "+r"(v[21]), "+r"(v[22]), "+r"(v[23]),
                 "+r"(v[24]), "+r"(v[25]), "+r"(v[26]), "+r"(v[27]), "+r"(v[28]), "+r"(v[29]),
                 "+r"(v[30]), "+r"(v[31])::"memory");
}
__device__ __forceinline__ void tmem_done(int (&v)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]),
                 "+r"(v[6]), "+r"(v[7]), "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]),
                 "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15])::"memory");
}

// ---- epilogue: one lane's channel, consecutive tokens --------------------------
struct Channel {
  int64_t n;
  bool in;
  float scale, bias;
};
__device__ __forceinline__ Channel channel_of(const LinParams& p, int64_t n) {
  Channel c;
  c.n = n;
  c.in = n < p.N;
  c.scale = c.in ? __ldg(p.ws + n) : 0.0f;
  c.bias = c.in && p.bias ? __ldg(p.bias + n) : 0.0f;
  return c;
}
// the scale of token t0 + lane, which the other lanes read by shuffle
__device__ __forceinline__ float token_scale(const LinParams& p, int64_t t0, int n) {
  const int lane = threadIdx.x & 31;
  return lane < n && t0 + lane < p.M ? __ldg(p.xs + t0 + lane) : 0.0f;
}
// kN tokens from t0; xs holds the scale of token t0 + at in lane `at`
template <typename T, int kN>
__device__ __forceinline__ void store_tokens(const LinParams& p, const Channel& c, int64_t t0,
                                             float xs, const int (&acc)[kN]) {
  T* y = static_cast<T*>(p.y) + t0 * p.ldy + c.n;
  const int64_t left = p.M - t0;  // (the same in the whole warp)
  if (left >= kN) {
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const float s = __shfl_sync(0xFFFFFFFFu, xs, i);
      if (c.in) y[0] = from_f32<T>(fmaf((float)acc[i], s * c.scale, c.bias));
      y += p.ldy;
    }
  } else {
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const float s = __shfl_sync(0xFFFFFFFFu, xs, i);
      if (c.in && i < left) y[0] = from_f32<T>(fmaf((float)acc[i], s * c.scale, c.bias));
      y += p.ldy;
    }
  }
}
template <int kN>
__device__ __forceinline__ void store_any(const LinParams& p, const Channel& c, int64_t t0,
                                          float xs, const int (&acc)[kN]) {
  if (p.dtype == SSMQ_F16)
    store_tokens<__half>(p, c, t0, xs, acc);
  else if (p.dtype == SSMQ_BF16)
    store_tokens<__nv_bfloat16>(p, c, t0, xs, acc);
  else
    store_tokens<float>(p, c, t0, xs, acc);
}
// NaN for `n` tokens from t0 of this lane's channel: the outputs that a call whose
// wait gave up does not finish
__device__ __forceinline__ void poison_tokens(const LinParams& p, const Channel& c, int64_t t0,
                                              int n) {
  const float nan = __int_as_float(0x7fffffff);
#pragma unroll 1
  for (int i = 0; i < n && t0 + i < p.M; ++i) {
    const int64_t at = (t0 + i) * p.ldy + c.n;
    if (!c.in) continue;
    if (p.dtype == SSMQ_F16)
      static_cast<__half*>(p.y)[at] = from_f32<__half>(nan);
    else if (p.dtype == SSMQ_BF16)
      static_cast<__nv_bfloat16*>(p.y)[at] = from_f32<__nv_bfloat16>(nan);
    else
      static_cast<float*>(p.y)[at] = nan;
  }
}
// The same values into a shared-memory tile [token][128 channels], at this lane's
// channel.
template <typename T>
__device__ __forceinline__ void stage_tokens(const Channel& c, float xs, const int (&acc)[32],
                                             uint32_t at) {
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    const float v = fmaf((float)acc[i], __shfl_sync(0xFFFFFFFFu, xs, i) * c.scale, c.bias);
    if constexpr (sizeof(T) == 4) {
      asm volatile("st.shared.f32 [%0], %1;" ::"r"(at + i * kRows * 4), "f"(v) : "memory");
    } else {
      const T h = from_f32<T>(v);
      asm volatile("st.shared.u16 [%0], %1;" ::"r"(at + i * kRows * 2),
                   "h"(*reinterpret_cast<const uint16_t*>(&h))
                   : "memory");
    }
  }
}
__device__ __forceinline__ void tma_store(const CUtensorMap* map, uint32_t src, int ch, int tok) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                   map),
               "r"(ch), "r"(tok), "r"(src)
               : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
// the shared memory of the stores so far may be written again
__device__ __forceinline__ void tma_stores_read() {
  asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
}

// ---- few tokens: 128 channels x kTok tokens per cluster, K split over its CTAs --
// Bound: the weight bytes (HBM).  The channel tiles alone are too few to pull
// the memory's bandwidth, so the CTAs of a cluster take consecutive parts of K
// of the same tile; each CTA then sums its share of the token columns from all
// parts (32-bit integers pushed through distributed shared memory: exact, no
// workspace, no second launch).  A wait that gives up raises a word in every CTA of the
// cluster; they then write NaN to the tile and wait for copies and MMAs in flight.
constexpr int kSplitThreads = 192;  // 4 epilogue warps, 1 TMA, 1 MMA
constexpr int kMaxSplit = 4;  // (clusters of 8 such CTAs waited for SMs: 12 us against 8)

template <int kTok>
struct SplitCfg {
  static constexpr int kStage = kOperand + kTok * kBlockK;
  // with a split: [part][channel][token column of the CTA], rows 16 bytes longer
  // than their columns (no bank conflicts)
  static int red(int split) { return split > 1 ? (kTok + 4 * split) * kRows * 4 : 0; }
  static constexpr int kBars = 256;              // barriers, TMEM address, abort word
  static constexpr int kMaxStages = 12;
  static constexpr int kCols = kTok < 32 ? 32 : kTok;
  static constexpr int kLd = kTok < 32 ? 16 : 32;  // token columns per TMEM load
  static int smem(int stages, int split) { return 1024 + kBars + stages * kStage + red(split); }
};

template <int kTok>
__global__ void __launch_bounds__(kSplitThreads)
    int8_linear_split_kernel(const __grid_constant__ CUtensorMap wmap,
                             const __grid_constant__ CUtensorMap xmap, const LinParams p,
                             const int split, const int stages) {
  using Cfg = SplitCfg<kTok>;
  constexpr int kLd = Cfg::kLd;
  extern __shared__ uint8_t raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~1023ull);
  uint64_t* full = reinterpret_cast<uint64_t*>(base + stages * Cfg::kStage);
  uint64_t* empty = full + Cfg::kMaxStages;
  uint64_t* done = empty + Cfg::kMaxStages;
  uint32_t* slot = reinterpret_cast<uint32_t*>(done + 1);
  volatile uint32_t* gave_up = slot + 1;
  int* red = reinterpret_cast<int*>(base + stages * Cfg::kStage + Cfg::kBars);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = split > 1 ? cta_rank() : 0;
  const int64_t tile = blockIdx.x / split;
  const int64_t ch0 = (tile % p.ch_tiles) * kRows, tok0 = (tile / p.ch_tiles) * kTok;
  const int kb0 = (int)((int64_t)p.kblocks * rank / split);
  const int kb1 = (int)((int64_t)p.kblocks * (rank + 1) / split);

  auto load = [&](int kb, int s) {
    const uint32_t bar = tc::smem_u32(full + s);
    const uint32_t dst = tc::smem_u32(base + s * Cfg::kStage);
    stream::expect_tx(full + s, Cfg::kStage);
    tma_load(dst, &wmap, kb * kBlockK, (int)ch0, bar);
    tma_load(dst + kOperand, &xmap, kb * kBlockK, (int)tok0, bar);
  };
  const int first = kb1 - kb0 < stages ? kb1 - kb0 : stages;  // loads without a wait
  if (warp == 4 && lane == 0) {
    prefetch_map(&wmap);
    prefetch_map(&xmap);
    for (int i = 0; i < stages; ++i) {
      tc::mbar_init(full + i, 1);
      tc::mbar_init(empty + i, 1);
    }
    tc::mbar_init(done, 1);
    *gave_up = 0;
    // the copies that need no empty stage start before the CTA meets
    for (int i = 0; i < first; ++i) load(kb0 + i, i);
  }
  if (warp == 5) tc::tmem_alloc(slot, Cfg::kCols);
  tc::fence_before();
  __syncthreads();
  if (split > 1) cluster_sync();  // every CTA of the cluster runs before one pushes to it
  tc::fence_after();
  const uint32_t tmem = *slot;
  auto give_up = [&] {  // (after the barrier above: the other CTAs' words are set up)
    *gave_up = 1;
    for (int r = 0; split > 1 && r < split; ++r)
      store_remote(mapa(tc::smem_u32(slot + 1), (uint32_t)r), 1u);
  };

  int issued = 0;  // stages filled
  if (warp == 4 && lane == 0) {
    int s = 0;
    uint32_t phase = 0;
    int kb = kb0 + first;
    for (; kb < kb1; ++kb) {
      if (!tc::mbar_wait(empty + s, phase, p.wait_limit)) {
        give_up();
        break;
      }
      load(kb, s);
      if (++s == stages) s = 0, phase ^= 1u;
    }
    issued = kb - kb0;
  } else if (warp == 5 && lane == 0) {
    constexpr uint32_t idesc = idesc_i8(kRows, kTok);
    int s = 0;
    uint32_t phase = 0;
    for (int kb = kb0; kb < kb1; ++kb) {
      if (!tc::mbar_wait(full + s, phase, kWaitLimit)) {
        give_up();
        break;
      }
      tc::fence_after();
      const uint32_t a = tc::smem_u32(base + s * Cfg::kStage);
      const uint64_t ad = sw128_desc(a), bd = sw128_desc(a + kOperand);
#pragma unroll
      for (int q = 0; q < kBlockK / 32; ++q)
        mma_i8<1>(tmem, ad + 2 * q, bd + 2 * q, idesc, kb > kb0 || q > 0);
      tc::mma_commit(empty + s);
      if (++s == stages) s = 0, phase ^= 1u;
    }
    tc::mma_commit(done);
  }
  __syncwarp();

  const int per = kTok / split;  // token columns that a CTA finishes: a multiple of 4
  const int pitch = per + 4;
  const int ch = (warp & 3) * 32 + lane;
  const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
  Channel c;
  if (warp < 4) {
    c = channel_of(p, ch0 + ch);
    float xs = split == 1 ? token_scale(p, tok0, kLd) : 0.0f;
    const bool ok = __all_sync(0xFFFFFFFFu, tc::mbar_wait(done, 0, p.wait_limit));
    if (!ok && lane == 0) give_up();
    tc::fence_after();
    for (int j = 0; j < kTok; j += kLd) {
      if (!ok || tok0 + j >= p.M) break;
      int v[kLd];
      tmem_get(lanes + j, v);
      tmem_done(v);
      if (split == 1) {
        const float next = token_scale(p, tok0 + j + kLd, kLd);
        store_any(p, c, tok0 + j, xs, v);
        xs = next;
      } else {
        // column j goes to CTA j / per
        const uint32_t local = tc::smem_u32(red + ((int)rank * kRows + ch) * pitch);
#pragma unroll
        for (int i = 0; i < kLd; i += 4) {
          const int owner = (j + i) / per, at = (j + i) % per;
          asm volatile("st.shared::cluster.v4.s32 [%0], {%1, %2, %3, %4};" ::"r"(
                           mapa(local + (uint32_t)at * 4, (uint32_t)owner)),
                       "r"(v[i]), "r"(v[i + 1]), "r"(v[i + 2]), "r"(v[i + 3])
                       : "memory");
        }
      }
    }
  }
  if (split > 1) {
    // this CTA's columns: their scales arrive while the others finish
    const int64_t mine = tok0 + (int64_t)rank * per;
    float xs[kTok >= 64 ? 2 : 1];
#pragma unroll
    for (int i = 0; i < (kTok >= 64 ? 2 : 1); ++i)
      xs[i] = warp < 4 ? token_scale(p, mine + 32 * i, per - 32 * i) : 0.0f;
    cluster_sync();
    if (warp < 4) {
#pragma unroll 1
      for (int j = 0; j < per; j += 4) {
        if (mine + j >= p.M) break;
        int acc[4] = {0, 0, 0, 0};
#pragma unroll 4
        for (int r = 0; r < split; ++r) {
          const int4 q = *reinterpret_cast<const int4*>(red + (r * kRows + ch) * pitch + j);
          acc[0] += q.x, acc[1] += q.y, acc[2] += q.z, acc[3] += q.w;
        }
        // (the scales of columns j .. j + 3 to lanes 0 .. 3)
        const float s = kTok >= 64 && j >= 32 ? xs[kTok >= 64 ? 1 : 0] : xs[0];
        store_any(p, c, mine + j, __shfl_sync(0xFFFFFFFFu, s, (lane + j) & 31), acc);
      }
    }
  }
  tc::fence_before();
  __syncthreads();
  if (*gave_up) {  // (raised in front of the barriers above)
    if (warp == 4 && lane == 0)  // the last `stages` copies are the only ones still open
      for (int j = issued > stages ? issued - stages : 0; j < issued; ++j)
        tc::mbar_wait(full + j % stages, (uint32_t)(j / stages) & 1u, kWaitLimit);
    if (warp == 5) tc::mbar_wait(done, 0, kWaitLimit);
    if (warp < 4) poison_tokens(p, c, tok0 + (int64_t)rank * per, per);
    __syncwarp();
  }
  if (warp == 5) tc::tmem_dealloc(tmem, Cfg::kCols);
  if (threadIdx.x == 0 && *gave_up) flag_status(p.status, SSMQ_DEV_TIMEOUT);
}

// ---- many tokens: 256 channels x 256 tokens per CTA pair, persistent -----------
// Bound: the tensor cores.  The two SMs of a pair share one 256 x 256 tile:
// each brings 128 channels and 128 tokens per K block (half the operand
// traffic per MMA of two separate 128 x 256 tiles), the leader issues the
// MMAs of both.  Accumulators are double-buffered in TMEM (2 x 256 columns),
// so eight warps per CTA write tile i (through shared memory by TMA, 256-byte rows,
// where y's rows are whole 16-byte pieces) while the MMAs of tile i + 1 run (four were
// slower than the MMAs: 206 against 126 us of MMAs at 16384 x 2560 x 5120).
// A wait that gives up raises a word in both CTAs.  Each role then ends by itself (no
// accumulator is handed on that is not complete), the epilogue writes NaN to the tiles
// it has left, and behind the pair's last barrier the copies and MMAs in flight are
// waited for, before shared and tensor memory go.
constexpr int kPairThreads = 384;  // warp 0 TMA, 1 MMA, 2 TMEM, 4-11 epilogue
constexpr int kPairStages = 5;  // (4 to 7 measured the same)
constexpr int kPairStage = 2 * kOperand;
constexpr int kPairTok = 256, kPairCh = 256;
// epilogue staging per half tile: 128 channels of 128 tokens in 16 bits, or of 64
// in 32 bits
constexpr int kHalfStage = 128 * kRows * 2;
constexpr int kPairSmem = 1024 + kPairStages * kPairStage + 2 * kHalfStage + 256;
static_assert(kPairSmem <= 227 * 1024, "shared memory");

// Tile i -> (channel tile, token tile): channels fastest inside a group of
// p.group channel tiles, so that the tiles in flight share tokens and the
// group's weights stay in L2.
__device__ __forceinline__ void tile_at(const LinParams& p, int64_t i, int64_t& ch, int64_t& tok) {
  const int64_t per = p.group * p.tok_tiles;
  const int64_t g = i / per, r = i % per;
  const int64_t left = p.ch_tiles - g * p.group;
  const int64_t w = left < p.group ? left : p.group;
  ch = g * p.group + r % w;
  tok = r / w;
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads)
    int8_linear_pair_kernel(const __grid_constant__ CUtensorMap wmap,
                            const __grid_constant__ CUtensorMap xmap,
                            const __grid_constant__ CUtensorMap ymap, const LinParams p) {
  extern __shared__ uint8_t raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~1023ull);
  uint8_t* out = base + kPairStages * kPairStage;  // epilogue staging
  uint64_t* full = reinterpret_cast<uint64_t*>(out + 2 * kHalfStage);
  uint64_t* empty = full + kPairStages;
  uint64_t* acc_full = empty + kPairStages;  // [2]
  uint64_t* acc_empty = acc_full + 2;        // [2], the leader's collect both CTAs
  uint64_t* idle = acc_empty + 2;            // after a wait gave up: the MMAs are done
  uint32_t* slot = reinterpret_cast<uint32_t*>(idle + 1);
  volatile uint32_t* gave_up = slot + 1;
  // the leader's: stages filled by the other CTA
  volatile int64_t* other_uses = reinterpret_cast<volatile int64_t*>(slot + 2);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cta_rank();
  const int64_t tiles = p.tok_tiles * p.ch_tiles;
  const int64_t pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kPairStages; ++i) {
      tc::mbar_init(full + i, 1);
      tc::mbar_init(empty + i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(acc_full + i, 1);
      tc::mbar_init(acc_empty + i, 2 * 8);  // the epilogue warps of both CTAs
    }
    tc::mbar_init(idle, 1);
    *gave_up = 0;
  }
  if (warp == 2) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     tc::smem_u32(slot)),
                 "r"(512));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
  }
  tc::fence_before();
  cluster_sync();  // barriers of both CTAs exist
  tc::fence_after();
  const uint32_t tmem = *slot;
  auto give_up = [&] {  // (after the barrier above: the other CTA's word is set up)
    *gave_up = 1;
    store_remote(mapa(tc::smem_u32(slot + 1), rank ^ 1u), 1u);
  };

  int64_t uses = 0;  // stages filled by this CTA
  if (warp == 0 && lane == 0) {
    prefetch_map(&wmap);
    prefetch_map(&xmap);
    int64_t i = 0;  // stage uses
    bool ok = true;
    for (int64_t t = pair; t < tiles && ok; t += pairs) {
      int64_t ch, tok;
      tile_at(p, t, ch, tok);
      const int wrow = (int)(ch * kPairCh + rank * kRows);
      const int xrow = (int)(tok * kPairTok + rank * kRows);
      for (int kb = 0; kb < p.kblocks; ++kb, ++i) {
        const int s = (int)(i % kPairStages);
        if (i >= kPairStages &&
            !tc::mbar_wait(empty + s, (uint32_t)(i / kPairStages - 1) & 1u, p.wait_limit)) {
          ok = false;
          break;
        }
        const uint32_t bar = mapa(tc::smem_u32(full + s), 0);
        const uint32_t dst = tc::smem_u32(base + s * kPairStage);
        if (rank == 0) stream::expect_tx(full + s, 2 * kPairStage);
        tma_load_pair(dst, &wmap, kb * kBlockK, wrow, bar);
        tma_load_pair(dst + kOperand, &xmap, kb * kBlockK, xrow, bar);
      }
    }
    if (!ok) give_up();
    uses = i;
    if (rank == 1) store_remote64(mapa(tc::smem_u32(const_cast<int64_t*>(other_uses)), 0), uses);
  } else if (warp == 1 && lane == 0 && rank == 0) {
    constexpr uint32_t idesc = idesc_i8(kPairCh, kPairTok);
    int64_t i = 0;
    int64_t n = 0;  // tiles of this pair
    bool ok = true;
    for (int64_t t = pair; t < tiles; t += pairs, ++n) {
      const int b = (int)(n & 1);
      if (n >= 2 && !tc::mbar_wait(acc_empty + b, (uint32_t)(n / 2 - 1) & 1u, kWaitLimit)) {
        ok = false;
        break;
      }
      tc::fence_after();
      const uint32_t d = tmem + (uint32_t)b * kPairTok;
      for (int kb = 0; kb < p.kblocks; ++kb, ++i) {
        const int s = (int)(i % kPairStages);
        if (!tc::mbar_wait(full + s, (uint32_t)(i / kPairStages) & 1u, kWaitLimit)) {
          ok = false;
          break;
        }
        tc::fence_after();
        const uint32_t a = tc::smem_u32(base + s * kPairStage);
        const uint64_t ad = sw128_desc(a), bd = sw128_desc(a + kOperand);
#pragma unroll
        for (int q = 0; q < kBlockK / 32; ++q)
          mma_i8<2>(d, ad + 2 * q, bd + 2 * q, idesc, kb > 0 || q > 0);
        commit_pair(empty + s);
      }
      if (!ok) break;
      commit_pair(acc_full + b);
    }
    if (!ok) give_up();
  } else if (warp >= 4) {
    const int quarter = warp & 3;                  // TMEM lanes that the warp may read
    const int half = (warp - 4) / 4 * (kPairTok / 2);  // its token columns
    const uint32_t half_bar = 1 + (warp - 4) / 4;  // the half's four warps meet here
    const bool one = quarter == 0 && lane == 0;    // issues the half's stores
    int64_t n = 0, t = pair;
    for (; t < tiles; t += pairs, ++n) {
      const int b = (int)(n & 1);
      int64_t ch, tok;
      tile_at(p, t, ch, tok);
      const Channel c = channel_of(p, ch * kPairCh + rank * kRows + quarter * 32 + lane);
      const int64_t t0 = tok * kPairTok + half;
      float xs[kPairTok / 64];
#pragma unroll
      for (int q = 0; q < kPairTok / 64; ++q) xs[q] = token_scale(p, t0 + 32 * q, 32);
      // the half's warps go on together (they meet again below), and its staging is
      // free then; without staging each warp decides for itself
      bool ok = tc::mbar_wait(acc_full + b, (uint32_t)(n / 2) & 1u, p.wait_limit);
      if (p.tma_out) {
        if (one) tma_stores_read();
        ok = all_of(half_bar, 128, ok);
      } else {
        ok = __all_sync(0xFFFFFFFFu, ok);
      }
      if (!ok) {
        if (lane == 0) give_up();
        break;
      }
      tc::fence_after();
      const uint32_t src = tmem + (uint32_t)(b * kPairTok + half) + ((uint32_t)(quarter * 32) << 16);
      const uint32_t at = tc::smem_u32(out + (warp - 4) / 4 * kHalfStage);
      const int64_t ch0 = ch * kPairCh + rank * kRows;
      // the half's four warps meet: its staging is complete
      auto send_stage = [&](int64_t tok0) {
        tc::fence_async_smem();
        tc::named_sync(half_bar, 128);
        if (one && ch0 < p.N && tok0 < p.M) tma_store(&ymap, at, (int)ch0, (int)tok0);
      };
      int v[2][32];
      tmem_get(src, v[0]);
#pragma unroll
      for (int q = 0; q < kPairTok / 64; ++q) {
        tmem_done(v[q & 1]);
        if (q + 1 < kPairTok / 64) {
          tmem_get(src + 32 * (q + 1), v[(q + 1) & 1]);
        } else {  // the columns are in registers: the next tile's MMAs may start
          tc::fence_before();
          __syncwarp();
          if (lane == 0) arrive_remote(mapa(tc::smem_u32(acc_empty + b), 0));
        }
        const int col = quarter * 32 + lane;
        if (!p.tma_out) {
          if (t0 + 32 * q < p.M) store_any(p, c, t0 + 32 * q, xs[q], v[q & 1]);
        } else if (p.dtype == SSMQ_F32) {
          if (q == 2) {
            send_stage(t0);
            if (one) tma_stores_read();
            tc::named_sync(half_bar, 128);
          }
          stage_tokens<float>(c, xs[q], v[q & 1], at + ((q & 1) * 32 * kRows + col) * 4);
        } else if (p.dtype == SSMQ_F16) {
          stage_tokens<__half>(c, xs[q], v[q & 1], at + (q * 32 * kRows + col) * 2);
        } else {
          stage_tokens<__nv_bfloat16>(c, xs[q], v[q & 1], at + (q * 32 * kRows + col) * 2);
        }
      }
      if (p.tma_out) send_stage(p.dtype == SSMQ_F32 ? t0 + 64 : t0);
    }
    for (; t < tiles; t += pairs) {  // after a wait gave up
      int64_t ch, tok;
      tile_at(p, t, ch, tok);
      poison_tokens(p, channel_of(p, ch * kPairCh + rank * kRows + quarter * 32 + lane),
                    tok * kPairTok + half, kPairTok / 2);
    }
    if (one)  // the stores are done before the CTA leaves
      asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  }
  __syncwarp();
  tc::fence_before();
  cluster_sync();  // the pair's MMAs, copies and remote arrivals are done
  if (*gave_up) {  // (the same in both CTAs) or may still be in flight
    if (warp == 0 && lane == 0 && rank == 0) {
      // Both CTAs' copies count on the leader's barriers.  A stage that only one of
      // them filled is made to expect that one's bytes; the last kPairStages uses are
      // the only ones that can be open.
      const int64_t theirs = *other_uses, most = uses > theirs ? uses : theirs;
      for (int64_t j = most > kPairStages ? most - kPairStages : 0; j < most; ++j) {
        uint64_t* bar = full + j % kPairStages;
        if (j >= uses)
          stream::expect_tx(bar, kPairStage);
        else if (j >= theirs)
          complete_tx(bar, kPairStage);
        tc::mbar_wait(bar, (uint32_t)(j / kPairStages) & 1u, kWaitLimit);
      }
    }
    if (warp == 1 && lane == 0) {
      if (rank == 0) commit_pair(idle);
      tc::mbar_wait(idle, 0, kWaitLimit);
    }
    __syncwarp();
    cluster_sync();
  }
  if (warp == 2)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
  if (threadIdx.x == 0 && *gave_up) flag_status(p.status, SSMQ_DEV_TIMEOUT);
}

// ---- rows onto 16-byte boundaries -----------------------------------------------
// Operands whose base or stride TMA cannot take are copied once to rows of a
// multiple of 16 bytes (zero-padded): one aligned 16-byte store per thread,
// its bytes gathered from aligned 32-bit words (whose other bytes are dropped).
struct AlignJob {
  const int8_t* src;
  int64_t stride, rows;
  int8_t* dst;
};
__global__ void __launch_bounds__(256) align_rows_kernel(const AlignJob a, const AlignJob b,
                                                         int64_t len, int64_t pitch) {
  const int64_t per = pitch / 16;
  int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const bool second = i >= a.rows * per;  // one launch for both operands
  if (second) i -= a.rows * per;
  if (i >= (second ? b.rows : a.rows) * per) return;
  const int64_t r = i / per, c = (i % per) * 16;
  const int8_t* s = (second ? b.src : a.src) + r * (second ? b.stride : a.stride) + c;
  int8_t* dst = second ? b.dst : a.dst;
  uint32_t w[4] = {0, 0, 0, 0};
  if (c + 16 <= len) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(s);
    const int sh = (int)(at & 3) * 8;
    const uint32_t* q = reinterpret_cast<const uint32_t*>(at & ~(uintptr_t)3);
    if (sh == 0) {
#pragma unroll
      for (int k = 0; k < 4; ++k) w[k] = q[k];
    } else {
      // (the fifth word holds bytes of this row: the piece is not aligned)
      uint32_t v = q[0];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t u = q[k + 1];
        w[k] = __funnelshift_r(v, u, sh);
        v = u;
      }
    }
  } else {
    for (int k = 0; k < 16; ++k)
      if (c + k < len) w[k >> 2] |= (uint32_t)(uint8_t)s[k] << (8 * (k & 3));
  }
  *reinterpret_cast<uint4*>(dst + r * pitch + c) = make_uint4(w[0], w[1], w[2], w[3]);
}

__global__ void __launch_bounds__(256) bias_rows_kernel(const LinParams p) {
  const int64_t n = p.M * p.N;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
    const int64_t t = i / p.N, c = i % p.N;
    const float v = p.bias ? p.bias[c] : 0.0f;
    if (p.dtype == SSMQ_F16)
      static_cast<__half*>(p.y)[t * p.ldy + c] = __float2half_rn(v);
    else if (p.dtype == SSMQ_BF16)
      static_cast<__nv_bfloat16*>(p.y)[t * p.ldy + c] = __float2bfloat16_rn(v);
    else
      static_cast<float*>(p.y)[t * p.ldy + c] = v;
  }
}

// ---- host ----------------------------------------------------------------------
int64_t pitch_of(int64_t k) { return (k + 15) / 16 * 16; }
size_t up256(size_t n) { return (n + 255) / 256 * 256; }
bool tma_rows(const void* p, int64_t rows, int64_t stride) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && (rows <= 1 || stride % 16 == 0);
}

cudaError_t encode(CUtensorMap* map, const void* p, int64_t rows, int64_t k, int64_t stride,
                   int box_rows) {
  const cuuint64_t dims[2] = {(cuuint64_t)k, (cuuint64_t)rows};
  // (one row: its stride is never used, but has to be a multiple of 16)
  const cuuint64_t strides[1] = {(cuuint64_t)(rows <= 1 ? pitch_of(k) : stride)};
  const cuuint32_t box[2] = {(cuuint32_t)kBlockK, (cuuint32_t)box_rows};
  return encode_tiled(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, p, dims, strides, box,
                      CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
}

// Which kernel, tile and split: the smallest estimate of the time beyond the
// start that all share.  Measured on one B200 (us, device): a CTA takes in its
// operands at about 92 KB/us; exchanging parts of K costs 1.7 + 0.035 per token
// column; a round of the pair kernel costs 0.36 per 128 bytes of K, plus 1.6.
// Tokens x channels x K, the tile taken against the next best: 512 x 4096 x 4096
// 128 columns 14.0, pairs 16.0; 1024 x 4096 x 4096 pairs 17.0, 128 columns 19.0;
// 256 x 4096 x 1024 64 columns 6.5, 128 columns and 2 parts 12.7; 64 x 4096 x 8192
// 64 columns and 4 parts 13.6, 32 and 2 parts 15.5; 200 x 1000 x 1024 16 columns
// 5.6, 32 columns and 2 parts 7.4.
struct Plan {
  bool pair;
  int tok, split;
};
Plan plan_for(int64_t M, int64_t N, int kblocks, int sms) {
  Plan best = {false, 16, 1};
  double least = 1e300;
  const int64_t ch = (N + kRows - 1) / kRows;
  for (int tok = 16; tok <= 128; tok *= 2) {
    if (tok > 16 && tok >= 2 * M) break;  // (half the columns would be idle)
    const int64_t tiles = ch * ((M + tok - 1) / tok);
    for (int split = 1; split <= kMaxSplit && kblocks >= 4 * split; split *= 2) {
      if (split > 1 && tiles * split > sms) break;
      const double bytes = (double)((kblocks + split - 1) / split) * (kRows + tok) * kBlockK;
      const double fill = (double)(tiles * split) / sms;
      const double us = bytes / 92e3 * (fill > 1 ? fill : 1) + (split > 1 ? 1.7 + 0.035 * tok : 0);
      if (us < least) least = us, best = {false, tok, split};
    }
  }
  const int64_t pairs = ((M + kPairTok - 1) / kPairTok) * ((N + kPairCh - 1) / kPairCh);
  const int64_t rounds = (pairs + sms / 2 - 1) / (sms / 2);
  if (M > 128 && 1.6 + 0.36 * (double)rounds * kblocks < least) best.pair = true;
  return best;
}

template <int kTok>
cudaError_t launch_split(const CUtensorMap& wmap, const CUtensorMap& xmap, LinParams p, int split,
                         cudaStream_t st) {
  using Cfg = SplitCfg<kTok>;
  p.ch_tiles = (p.N + kRows - 1) / kRows;
  p.tok_tiles = (p.M + kTok - 1) / kTok;
  const int64_t tiles = p.ch_tiles * p.tok_tiles;
  if (tiles > 0x7fffffff / kMaxSplit) return cudaErrorInvalidConfiguration;
  // One CTA per SM takes all the stages that fit (or that its K needs); several
  // share the shared memory two to an SM.
  const int room = (tiles * split <= sm_count() ? 224 : 110) * 1024;
  int stages = (room - Cfg::smem(0, split)) / Cfg::kStage;
  const int need = (p.kblocks + split - 1) / split;
  stages = stages < Cfg::kMaxStages ? stages : Cfg::kMaxStages;
  stages = stages < need ? stages : need;
  stages = stages < 2 ? 2 : stages;
  const int smem = Cfg::smem(stages, split);
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(int8_linear_split_kernel<kTok>),
                                   227 * 1024, done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(tiles * split));
  cfg.blockDim = dim3(kSplitThreads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)split;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = split > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, int8_linear_split_kernel<kTok>, wmap, xmap, p, split, stages);
}

}  // namespace

size_t int8_linear_workspace_bytes(const ssmq_linear_args& a) {
  size_t n = 0;
  if (a.tokens <= 0 || a.out_features <= 0 || a.in_features <= 0) return 0;
  if (!tma_rows(a.x, a.tokens, a.x_stride))
    n += up256((size_t)a.tokens * pitch_of(a.in_features));
  if (!tma_rows(a.w, a.out_features, a.w_stride))
    n += up256((size_t)a.out_features * pitch_of(a.in_features));
  return n;
}

cudaError_t launch_int8_linear(const ssmq_linear_args& a, void* ws, cudaStream_t st) {
  LinParams p = {};
  p.M = a.tokens;
  p.N = a.out_features;
  p.kblocks = (int)((a.in_features + kBlockK - 1) / kBlockK);
  p.xs = a.x_scale;
  p.ws = a.w_scale;
  p.bias = a.bias;
  p.y = a.y;
  p.ldy = a.y_stride;
  p.dtype = a.dtype;
  p.status = a.status;
  p.wait_limit = stream::wait_limit();
  if (p.kblocks == 0) {
    const int64_t n = (p.M * p.N + 255) / 256, most = (int64_t)sm_count() * 8;
    bias_rows_kernel<<<(unsigned)(n < most ? n : most), 256, 0, st>>>(p);
    return cudaGetLastError();
  }
  const int8_t* x = a.x;
  const int8_t* w = a.w;
  int64_t xst = a.x_stride, wst = a.w_stride;
  const int64_t pitch = pitch_of(a.in_features);
  uint8_t* room = static_cast<uint8_t*>(ws);
  cudaError_t e;
  AlignJob jobs[2] = {};
  auto job = [&](AlignJob& j, const int8_t*& t, int64_t& stride, int64_t rows) {
    if (tma_rows(t, rows, stride)) return;
    j = AlignJob{t, stride, rows, reinterpret_cast<int8_t*>(room)};
    room += up256((size_t)rows * pitch);
    t = j.dst;
    stride = pitch;
  };
  job(jobs[0], x, xst, p.M);
  job(jobs[1], w, wst, p.N);
  if (const int64_t n = (jobs[0].rows + jobs[1].rows) * (pitch / 16)) {
    align_rows_kernel<<<(unsigned)((n + 255) / 256), 256, 0, st>>>(jobs[0], jobs[1], a.in_features,
                                                                   pitch);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }

  const int sms = sm_count();
  const Plan plan = plan_for(p.M, p.N, p.kblocks, sms);
  const int tok = plan.pair ? kRows : plan.tok;
  CUtensorMap wmap, xmap;
  if ((e = encode(&wmap, w, p.N, a.in_features, wst, kRows)) != cudaSuccess) return e;
  if ((e = encode(&xmap, x, p.M, a.in_features, xst, tok)) != cudaSuccess) return e;
  if (!plan.pair) {
    switch (tok) {
      case 16: return launch_split<16>(wmap, xmap, p, plan.split, st);
      case 32: return launch_split<32>(wmap, xmap, p, plan.split, st);
      case 64: return launch_split<64>(wmap, xmap, p, plan.split, st);
      default: return launch_split<128>(wmap, xmap, p, plan.split, st);
    }
  }
  p.tok_tiles = (p.M + kPairTok - 1) / kPairTok;
  p.ch_tiles = (p.N + kPairCh - 1) / kPairCh;
  p.group = 16;
  static std::atomic<uint64_t> done{0};
  e = allow_smem(reinterpret_cast<const void*>(int8_linear_pair_kernel), kPairSmem, done);
  if (e != cudaSuccess) return e;
  CUtensorMap ymap = {};
  const int esz = p.dtype == SSMQ_F32 ? 4 : 2;
  // (a TMA store writes whole 16-byte pieces of a row: N has to end with one)
  if (rows16(p.y, p.ldy, esz) && p.N * esz % 16 == 0 && p.ldy < ((int64_t)1 << 36)) {
    const cuuint64_t dims[2] = {(cuuint64_t)p.N, (cuuint64_t)p.M};
    const cuuint64_t strides[1] = {(cuuint64_t)p.ldy * esz};
    const cuuint32_t box[2] = {(cuuint32_t)kRows, esz == 4 ? 64u : 128u};
    p.tma_out = encode_tiled(&ymap,
                             esz == 4 ? CU_TENSOR_MAP_DATA_TYPE_UINT32
                                      : CU_TENSOR_MAP_DATA_TYPE_UINT16,
                             2, p.y, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_NONE,
                             CU_TENSOR_MAP_L2_PROMOTION_NONE) == cudaSuccess;
  }
  const int64_t pair_tiles = p.tok_tiles * p.ch_tiles;
  const int64_t pairs = pair_tiles < sms / 2 ? pair_tiles : sms / 2;
  int8_linear_pair_kernel<<<(unsigned)(2 * pairs), kPairThreads, kPairSmem, st>>>(wmap, xmap, ymap,
                                                                                  p);
  return cudaGetLastError();
}

}  // namespace ssmq
