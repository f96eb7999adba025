// Building blocks of the gated recurrence h_t = f_t h_{t-1} + (1 - f_t) v_t:
// the tile of one CTA, its loads, and the exchange of carried states between
// the CTAs of a cluster.
//
// A CTA owns a block of channels and, per round, one tile of consecutive steps:
// kLanes lanes hold two channels each, every thread kSteps consecutive steps of
// its channels, so a warp holds 32 / kLanes segments and the CTA kWarps times as
// many.  A segment acts on the state entering it as h -> A h + B; (A, B) of
// segments, warps and CTAs compose in step order.  The CTAs of a cluster hold
// consecutive tiles and push their (A, B) into each other's shared memory; one
// exchange per round replaces a second pass over the data or a spin on global
// memory.
#pragma once

#include "internal.h"
#include "stream.cuh"
#include "tc.cuh"
#include "tma_map.h"
#include "vec8.cuh"

namespace ssmq {
namespace gated {

constexpr int kMaxCluster = 16;  // CTAs along time (above 8: non-portable)
constexpr uint32_t kWaitLimit = 1u << 20;

// How a tile's inputs reach shared memory.
enum {
  kTma = 0,    // whole tiles by TMA: rows on 16-byte boundaries
  kPairs = 1,  // each thread its own pairs of channels
  kSingle = 2  // rows on any element: its own channels one by one, or 16-bit ones as
               // the aligned words they lie in, shared by the lanes of a row
};

template <int kWarps_, int kSteps_, int kLanes_>
struct Tile {
  static constexpr int kWarps = kWarps_, kSteps = kSteps_, kLanes = kLanes_;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kChannels = 2 * kLanes;
  static constexpr int kSubs = 32 / kLanes;  // segments per warp
  static constexpr int kLen = kWarps * kSubs * kSteps;
  static_assert(kLen % kGatedStateSteps == 0, "saved states at tile starts");
  static_assert(kGatedStateSteps % kSteps == 0, "saved states at segment starts");
};

// The tile of a mode.  With TMA four warps of sixteen steps: the exchange between
// segments is per thread, and eight warps of eight steps spend more on it than on
// the steps (forward, 8 x 2048 x 1536 binary16, gated: 53 us against 45; gradient,
// 4 x 4096 x 5120 bfloat16: 264 against 250).  Where the threads copy for
// themselves, eight warps of eight: twice the threads have copies in flight
// (gradient, 5 x 1023 x 333 binary32: 31 us against 20).
template <int kMode, int kLanes>
using ModeTile = Tile<kMode == kTma ? 4 : 8, kMode == kTma ? 16 : 8, kLanes>;

struct Rows {
  void* p;
  int64_t bs, rs;
};
inline Rows rows_of(const ssmq_rows& r) { return Rows{r.p, r.batch_stride, r.row_stride}; }

// two channels of one row
template <typename T>
struct Pair {
  uint32_t w;
};
template <>
struct Pair<float> {
  float2 w;
};
template <typename T>
__device__ __forceinline__ float2 pair_f32(Pair<T> p) { return unpack2<T>(p.w); }
template <>
__device__ __forceinline__ float2 pair_f32<float>(Pair<float> p) { return p.w; }

// Elements p[0] and p[next] (kVec: one store of a pair).
template <typename T, bool kVec>
__device__ __forceinline__ void store_pair(T* p, int next, float2 v, bool in0, bool in1) {
  if constexpr (kVec) {
    if (in0) {
      if constexpr (sizeof(T) == 4)
        *reinterpret_cast<float2*>(p) = v;
      else
        *reinterpret_cast<uint32_t*>(p) = pack2<T>(v.x, v.y);
    }
  } else {
    if (in0) p[0] = from_f32<T>(v.x);
    if (in1) p[next] = from_f32<T>(v.y);
  }
}

struct Maps {
  CUtensorMap m[4];
};

// Staged inputs: kBufs tiles of kTensors tensors in shared memory, filled ahead
// of the round that reads them, so that no register holds a load in flight.
// kTma: one thread fetches whole tiles ([row][channel]); rows and channels
// beyond the tensor read as zero.  Otherwise every thread copies the pairs of
// its own steps into slots of its own ([step][thread]), or the lanes of a row its
// words together ([step][row group][word]).  Either way a thread reads only its
// own steps and channels.  kDirect: copies of 16-bit channels and of pairs go
// through registers, not as asynchronous copies of 4 bytes, which the forward kernel
// with its many warps does not need (8 x 2048 x 1538 binary16, gated: 108 us against
// 67; odd rows, 1537: 108 against 84; the gradient's odd rows: 188 against 234).
template <typename T, int kTensors, int kMode, typename TileT, int kBufs_, bool kDirect>
struct Stage {
  static constexpr int kThreads = TileT::kThreads, kSteps = TileT::kSteps;
  static constexpr int kBufs = kBufs_;
  static constexpr int kLanes = TileT::kLanes;
  // 16-bit rows on any element: a row's kLanes + 1 words hold its 2 kLanes channels
  // from either half of the first word on
  static constexpr bool kWords = kMode == kSingle && sizeof(T) == 2 && !kDirect;
  // channels of a thread's pair: side by side, or kLanes apart
  static constexpr int kNext = kMode == kSingle && !kWords ? kLanes : 1;
  static constexpr int kStepBytes = kMode == kTma ? TileT::kChannels * (int)sizeof(T)
                                    : kWords      ? kThreads / kLanes * (kLanes + 1) * 4
                                                  : 2 * kThreads * (int)sizeof(T);
  static constexpr int kTensorBytes = (kMode == kTma ? TileT::kLen : kSteps) * kStepBytes;
  static constexpr int kBytes = kBufs * kTensors * kTensorBytes;
  uint8_t* base;  // of this thread's pairs
  uint32_t halves[2] = {0, 0};  // kWords: bit j, the half word that even (odd) rows of tensor j
                                // start in (segments start at even rows)
  int channels = 0;             // kWords: channels of the block
  __device__ __forceinline__ explicit Stage(uint8_t* smem) {
    const int lane = threadIdx.x & 31;
    if constexpr (kMode == kTma) {
      const int row = ((int)(threadIdx.x >> 5) * TileT::kSubs + lane / kLanes) * kSteps;
      base = smem + row * kStepBytes + (lane % kLanes) * 2 * (int)sizeof(T);
    } else if constexpr (kWords) {
      base = smem + ((int)threadIdx.x / kLanes * (kLanes + 1) + lane % kLanes) * 4;
    } else {
      base = smem + threadIdx.x * 2 * (int)sizeof(T);
    }
  }
  // kWords: where the rows of a tensor start (p: its channel block's first row)
  __device__ __forceinline__ void rows_at(int tensor, const T* p, int64_t rs) {
    if constexpr (kWords) {
      const uint32_t even = (uint32_t)(reinterpret_cast<uintptr_t>(p) >> 1) & 1u;
      halves[0] |= even << tensor;
      halves[1] |= (even ^ ((uint32_t)rs & 1u)) << tensor;
    }
  }
  __device__ __forceinline__ uint8_t* at(int buf, int tensor) const {
    return base + (buf * kTensors + tensor) * kTensorBytes;
  }
  __device__ __forceinline__ float2 get(int buf, int tensor, int i) const {
    if constexpr (kWords) {
      const uint32_t* w = reinterpret_cast<const uint32_t*>(at(buf, tensor) + i * kStepBytes);
      const uint32_t half = (halves[i & 1] >> tensor) & 1u;
      return pair_f32<T>(Pair<T>{__funnelshift_r(w[0], w[1], 16 * half)});
    }
    return pair_f32<T>(*reinterpret_cast<const Pair<T>*>(at(buf, tensor) + i * kStepBytes));
  }
  // kTma: the tile at (channel c, step t, sequence s) of one tensor
  static __device__ __forceinline__ void fetch_tile(uint8_t* smem, int buf, int tensor,
                                                    const CUtensorMap* map, int c, int t, int s,
                                                    uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], "
        "[%1, {%2, %3, %4}], [%5];" ::"r"(
            tc::smem_u32(smem + (buf * kTensors + tensor) * kTensorBytes)),
        "l"(map), "r"(c), "r"(t), "r"(s), "r"(tc::smem_u32(bar))
        : "memory");
  }
  // the other modes: rows 0 .. left - 1 of the thread's steps, zeros behind
  // them.  p: the thread's first channel (lanes without one have it clamped to
  // channel 0), for kWords the block's.
  __device__ __forceinline__ void fetch(int buf, int tensor, const T* p, int64_t rs, int next,
                                        int left) const {
    if constexpr (kDirect && (kMode == kPairs || sizeof(T) == 2)) {
      uint8_t* o = at(buf, tensor);
      Pair<T> r[kSteps];
      if constexpr (kMode == kPairs) {
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
          const T* src = p + i * rs;
          r[i] = Pair<T>{};
          if (i < left) r[i] = *reinterpret_cast<const Pair<T>*>(src);
        }
      } else {
        const uint16_t* u = reinterpret_cast<const uint16_t*>(p);
        if (left == kSteps) {  // (without branches between the loads)
#pragma unroll
          for (int i = 0; i < kSteps; ++i)
            r[i].w = (uint32_t)u[i * rs] | ((uint32_t)u[i * rs + next] << 16);
        } else {
#pragma unroll
          for (int i = 0; i < kSteps; ++i) {
            r[i] = Pair<T>{};
            if (i < left) r[i].w = (uint32_t)u[i * rs] | ((uint32_t)u[i * rs + next] << 16);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < kSteps; ++i) *reinterpret_cast<Pair<T>*>(o + i * kStepBytes) = r[i];
      return;
    }
    const uint32_t dst = tc::smem_u32(at(buf, tensor));
    if constexpr (kWords) {
      // words that hold a channel of the row; the half beside it (another channel, or at
      // the tensor's ends what lies beside it in that word) is dropped
      const int l = (int)threadIdx.x % kLanes;
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        const int half = (int)(halves[i & 1] >> tensor) & 1;
        const T* src = p + i * rs - half + 2 * l;
        copy4(dst + i * kStepBytes, src, i < left && 2 * l - half < channels);
        if (l == kLanes - 1)
          copy4(dst + i * kStepBytes + 4, src + 2, i < left && 2 * kLanes - half < channels);
      }
    } else {
      constexpr int kN = kMode == kPairs ? 1 : 2;  // copies per pair
      constexpr int kCopy = 2 * (int)sizeof(T) / kN;
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        const int bytes = i < left ? kCopy : 0;
#pragma unroll
        for (int j = 0; j < kN; ++j)
          asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(
                           dst + i * kStepBytes + j * kCopy),
                       "l"(p + i * rs + j * next), "n"(kCopy), "r"(bytes)
                       : "memory");
      }
    }
  }
  // four bytes, or (nothing read) zeros
  static __device__ __forceinline__ void copy4(uint32_t dst, const T* src, bool on) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src),
                 "r"(on ? 4 : 0)
                 : "memory");
  }
  // zeros in the thread's steps from `left` on: tiles by TMA bring the rows
  // behind a sequence's end, and no tile brings those in front of its start
  __device__ __forceinline__ void clear(int buf, int left) const {
    for (int j = 0; j < kTensors; ++j)
      for (int i = left; i < kSteps; ++i)
        *reinterpret_cast<Pair<T>*>(at(buf, j) + i * kStepBytes) = Pair<T>{};
    // (a later tile's copy into this buffer comes after these stores)
    tc::fence_async_smem();
  }
  static __device__ __forceinline__ void commit() {
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  // all but the newest kBufs - 1 groups have landed
  static __device__ __forceinline__ void wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(kBufs - 1) : "memory");
    if constexpr (kWords) __syncwarp();  // (the row's other lanes' words too)
  }
};
// rows of the segment at t0 that lie before the end, at most `steps`
__device__ __forceinline__ int rows_left(int64_t end, int64_t t0, int steps) {
  const int64_t n = end - t0;
  return n < 0 ? 0 : (n < steps ? (int)n : steps);
}

// e = exp(-g), r = 1 / (1 + e).  The smaller of f and n = 1 - f is r for g < 0, else
// e r, to a few ulps and the rounding of the exponent (|g| 2^-23); the larger is 1
// minus it (at most half an ulp off), not the approximate reciprocal, whose ulp a
// long memory would accumulate.  g = -inf: e = inf, f = 0, n = 1; a NaN g makes both
// NaN.
__device__ __forceinline__ void gate2(float2 g, float2& f, float2& n) {
  const float2 x = fmul2(g, make_float2(-kLog2e, -kLog2e));
  const float2 e = make_float2(ex2_sfu(x.x), ex2_sfu(x.y));
  const float2 one = make_float2(1.0f, 1.0f);
  const float2 d = fadd2(one, e);
  const float2 r = make_float2(rcp_sfu(d.x), rcp_sfu(d.y));
  const float2 er = fmul2(e, r);  // (g < 0: not used)
  const float2 not_r = fsub2(one, r), not_er = fsub2(one, er);
  const bool neg0 = g.x < 0.0f, neg1 = g.y < 0.0f;
  f = make_float2(neg0 ? r.x : not_er.x, neg1 ? r.y : not_er.y);
  n = make_float2(neg0 ? not_r.x : er.x, neg1 ? not_r.y : er.y);
}
__device__ __forceinline__ float2 sigmoid2(float2 z) {
  const float2 x = fmul2(z, make_float2(-kLog2e, -kLog2e));
  const float2 d = fadd2(make_float2(1.0f, 1.0f), make_float2(ex2_sfu(x.x), ex2_sfu(x.y)));
  return make_float2(rcp_sfu(d.x), rcp_sfu(d.y));
}

// ---- cluster ---------------------------------------------------------------
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Barriers at both ends of the kernel.  (Inside, states travel by st.async with
// an mbarrier at the receiver: a cluster barrier with release semantics would
// wait for the round's stores to global memory as well.)
__device__ __forceinline__ void cluster_meet() {
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
}
// 16 bytes into the same shared-memory location of CTA `rank` of the cluster,
// counted on the same barrier there
__device__ __forceinline__ void push_f4(float4* local, uint64_t* bar, uint32_t rank, float4 v) {
  uint32_t a, b;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(tc::smem_u32(local)), "r"(rank));
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(b) : "r"(tc::smem_u32(bar)), "r"(rank));
  asm volatile(
      "st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, "
      "[%5];" ::"r"(a),
      "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w), "r"(b)
      : "memory");
}

// Probes at most `limit` times; false means it gave up.
__device__ __forceinline__ bool wait_tile(uint64_t* bar, uint32_t parity, uint32_t limit) {
#pragma unroll 1
  for (uint32_t i = 0; i < limit; ++i)
    if (tc::mbar_try(bar, parity)) return true;
  return false;
}
// The same, acquiring what the other CTAs of the cluster wrote
__device__ __forceinline__ bool wait_cluster(uint64_t* bar, uint32_t parity, uint32_t limit) {
#pragma unroll 1
  for (uint32_t i = 0; i < limit; ++i) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(ok)
        : "r"(tc::smem_u32(bar)), "r"(parity), "r"(1000u)
        : "memory");
    if (ok) return true;
  }
  return false;
}

// (A, B) of two channels: {A0, A1, B0, B1}; h -> A h + B
__device__ __forceinline__ float2 apply(float4 m, float2 h) {
  return ffma2(make_float2(m.x, m.y), h, make_float2(m.z, m.w));
}
// first m, then n
__device__ __forceinline__ float4 compose(float4 m, float4 n) {
  const float2 a = fmul2(make_float2(m.x, m.y), make_float2(n.x, n.y));
  const float2 b = apply(n, make_float2(m.z, m.w));
  return make_float4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ float4 shfl_f4(float4 v, int src) {
  return make_float4(__shfl_sync(0xFFFFFFFFu, v.x, src), __shfl_sync(0xFFFFFFFFu, v.y, src),
                     __shfl_sync(0xFFFFFFFFu, v.z, src), __shfl_sync(0xFFFFFFFFu, v.w, src));
}

// What this CTA expects on `bar` less `bytes` that will not come.
__device__ __forceinline__ void complete_tx(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.complete_tx.relaxed.cluster.shared::cluster.b64 [%0], %1;" ::"r"(
                   tc::smem_u32(bar)),
               "r"(bytes)
               : "memory");
}
// the same word of shared memory in CTA `rank` of the cluster
__device__ __forceinline__ void store_remote(const uint32_t* local, uint32_t rank, uint32_t v) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(tc::smem_u32(local)), "r"(rank));
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}
__device__ __forceinline__ float2 nan2() {
  return make_float2(__int_as_float(0x7fffffff), __int_as_float(0x7fffffff));
}

template <typename TileT>
struct Shared {
  static constexpr int kWarps = TileT::kWarps, kLanes = TileT::kLanes;
  static constexpr int kMost = kLanes == 32 ? 8 : kMaxCluster;  // (wide blocks: portable clusters)
  float4 warp[2][kWarps][kLanes];
  float4 cta[2][kMost][kLanes];
  uint64_t bar[2];  // the maps of all CTAs of a round have arrived
  // After a wait gave up: the round at whose barrier the CTA left the exchange (kNever:
  // it has not), whether any CTA of the cluster gave up, the rounds that each has pushed.
  uint32_t leave_at, left, pushed[kMost];
};
constexpr uint32_t kNever = 0xFFFFFFFFu;

// Before the first round (every thread of the cluster).  All threads write the words:
// a branch for one of them here cost the gradient's word form 100 bytes of spills (307
// us against 271 at 8 x 2048 x 1537 binary16).
template <typename TileT>
__device__ __forceinline__ void carry_init(Shared<TileT>& sh, uint32_t size) {
  sh.leave_at = kNever;
  sh.left = 0;
  if (size == 1) return;
  if (threadIdx.x == 0) {
    tc::mbar_init(sh.bar, 1);
    tc::mbar_init(sh.bar + 1, 1);
  }
  cluster_sync();
}
// A thread whose wait gives up sets its word `late`.  At the CTA's next barrier all its
// threads learn of it (the word is set in every one) and leave the exchange: they wait
// for nothing, fetch and push nothing, and go through the rounds with a NaN state, so
// that what the CTA has not finished is NaN.  Returns that state.
template <typename TileT>
__device__ __forceinline__ float2 leave(Shared<TileT>& sh, int64_t k) {
  if (threadIdx.x == 0 && sh.leave_at == kNever) sh.leave_at = (uint32_t)k;
  return nan2();
}
// Behind the last round: nobody pushes to a CTA that has left.  A CTA that gave up has
// pushed k rounds only, so barriers may be open: the one that this CTA has armed for
// round k - 1, less what was never sent, and the one of round k, not armed yet, to which
// the others may have pushed.  (Round k - 2 had arrived before this CTA pushed round
// k - 1, and nobody pushes round k + 1 without this CTA's round k.)
template <typename TileT>
__device__ __forceinline__ void carry_done(Shared<TileT>& sh, int64_t rounds, uint32_t late) {
  uint32_t size;  // (read anew: no register holds it through the rounds)
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(size));
  if (size == 1) return;
  if (late) {
    for (uint32_t r = 0; r < size; ++r) store_remote(&sh.left, r, 1u);
    // (cluster_meet orders nothing by itself)
    asm volatile("fence.acq_rel.cluster;" ::: "memory");
  }
  __syncwarp();
  cluster_meet();
  if (*const_cast<volatile uint32_t*>(&sh.left) == 0) return;
  // (the same in every CTA of the cluster)
  if (threadIdx.x == 0) {
    const uint32_t k = sh.leave_at != kNever ? sh.leave_at : (uint32_t)rounds;
    for (uint32_t r = 0; r < size; ++r) store_remote(sh.pushed + cluster_rank(), r, k);
  }
  __syncwarp();
  cluster_sync();
  if (threadIdx.x == 0) {
    constexpr uint32_t kBytes = TileT::kLanes * (uint32_t)sizeof(float4);
    const uint32_t k = sh.pushed[cluster_rank()];
    uint32_t last = 0, now = 0;  // CTAs that pushed round k - 1, round k
    for (uint32_t r = 0; r < size; ++r) {
      last += sh.pushed[r] >= k;
      now += sh.pushed[r] > k;
    }
    if (k > 0) {
      uint64_t* bar = sh.bar + ((k - 1) & 1u);
      if (last < size) complete_tx(bar, (size - last) * kBytes);
      wait_tile(bar, ((k - 1) >> 1) & 1u, kWaitLimit);
    }
    if (now > 0) {
      uint64_t* bar = sh.bar + (k & 1u);
      stream::expect_tx(bar, now * kBytes);
      wait_tile(bar, (k >> 1) & 1u, kWaitLimit);
    }
  }
}

// State entering this thread's segment, from the segments' maps in step order
// (kReverse: in reverse step order, the last segment of the warp, warp and
// CTA first), and the state behind the whole round in h.  Every thread of the
// cluster calls it, round by round.  Buffers alternate between rounds: a CTA
// pushes round k + 2 only after it has every map of round k + 1, and a CTA pushes
// round k + 1 only when its threads are done with round k.  met() runs behind the
// CTA's barrier: every thread is done with the rounds before this one, and with
// what it read of this round before the call.  size and limit (of the waits) become 1
// and 0 where the CTA leaves the exchange.  kReverse: late is the CTA's already (a
// barrier lies between the round's waits and the call).
template <typename TileT, bool kReverse, typename Met>
__device__ __forceinline__ float2 carry_in(Shared<TileT>& sh, int64_t k, float4 m, float2& h,
                                           uint32_t rank, uint32_t& size, uint32_t& limit,
                                           uint32_t& late, Met met) {
  const int buf = (int)(k & 1);
  constexpr int kSubs = TileT::kSubs, kLanes = TileT::kLanes, kWarps = TileT::kWarps;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub0 = lane / kLanes, l = lane % kLanes;
  const int sub = kReverse ? kSubs - 1 - sub0 : sub0;  // position in processing order
  const int w = kReverse ? kWarps - 1 - warp : warp;
  // inclusive maps of the warp's segments
#pragma unroll
  for (int o = 1; o < kSubs; o <<= 1) {
    const int src = kReverse ? lane + o * kLanes : lane - o * kLanes;
    const float4 before = shfl_f4(m, src & 31);
    if (sub >= o) m = compose(before, m);
  }
  if (sub == kSubs - 1) sh.warp[buf][w][l] = m;
  float4 mine = make_float4(1.0f, 1.0f, 0.0f, 0.0f);  // the warp's segments before this one
  if constexpr (kSubs > 1) {
    const int src = kReverse ? lane + kLanes : lane - kLanes;
    const float4 before = shfl_f4(m, src & 31);
    if (sub > 0) mine = before;
  }
  if constexpr (kReverse)
    __syncthreads();
  else
    late = __syncthreads_or(late);
  if (late) {
    h = leave(sh, k);
    size = 1;
    limit = 0;
  }
  met();
  float4 pre = make_float4(1.0f, 1.0f, 0.0f, 0.0f), all = pre;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) {
    if (i == w) pre = all;
    all = compose(all, sh.warp[buf][i][l]);
  }
  float2 base = h;
  if (size > 1) {
    // warp i tells CTA i (and i + 8) of the cluster what this CTA's tile does to a state
    if (threadIdx.x == 0)
      stream::expect_tx(sh.bar + buf, size * kLanes * (uint32_t)sizeof(float4));
    if (sub0 == 0)
      for (uint32_t r = (uint32_t)warp; r < size; r += kWarps)
        push_f4(&sh.cta[buf][rank][l], sh.bar + buf, r, all);
    float2 s = h;
    if (!wait_cluster(sh.bar + buf, (uint32_t)(k >> 1) & 1u, limit)) {
      late = 1;
      s = base = nan2();
    }
    __syncwarp();
    // (four loads at a time, which do not wait on one another; size is 2, 4, 8 or 16,
    // and the entries of a cluster of 2 end after two)
    for (uint32_t r = 0; r < size; r += 4) {
      float4 e[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) e[i] = sh.cta[buf][r + i][l];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (r + i == rank) base = s;
        if (i < 2 || size > 2) s = apply(e[i], s);
      }
    }
    h = s;
  } else {
    h = apply(all, h);
  }
  return apply(mine, apply(pre, base));
}

// ---- host: launch shape -----------------------------------------------------
struct Shape {
  bool narrow;      // 16 channels per CTA instead of 64
  int cluster;
  unsigned grid;
  int64_t blocks;   // channel blocks per sequence
};
// (the tiles of all modes have the same sizes)
constexpr int kWideChannels = ModeTile<kTma, 32>::kChannels, kWideLen = ModeTile<kTma, 32>::kLen;
constexpr int kNarrowChannels = ModeTile<kTma, 8>::kChannels, kNarrowLen = ModeTile<kTma, 8>::kLen;
static_assert(ModeTile<kPairs, 32>::kLen == kWideLen && ModeTile<kPairs, 8>::kLen == kNarrowLen,
              "tiles");
// resident: CTAs that the GPU holds at once; fills: how many times the CTAs are to
// fill it (nearly: 0.85).
inline Shape shape_for(int64_t b, int64_t L, int64_t d, int64_t resident, int fills) {
  Shape s;
  // Time is split over a cluster until there are CTAs enough; where that leaves
  // the GPU partly idle, narrower channel blocks (32-byte rows of 16-bit
  // elements) and clusters of 16.
  auto pick = [&](int channels, int len, int most) {
    s.blocks = (d + channels - 1) / channels;
    const int64_t tiles = (L + len - 1) / len;
    s.cluster = 1;
    while (s.cluster < most && s.cluster < tiles &&
           b * s.blocks * s.cluster < resident * fills * 85 / 100)
      s.cluster *= 2;
    return b * s.blocks * s.cluster;
  };
  s.narrow = false;
  int64_t n = pick(kWideChannels, kWideLen, 8);
  if (n < resident * 85 / 100) {
    const Shape wide = s;
    s.narrow = true;
    const int64_t m = pick(kNarrowChannels, kNarrowLen, kMaxCluster);
    if (m <= n || L <= kNarrowLen / 2) s = wide;
    else n = m;
  }
  s.grid = (unsigned)n;
  return s;
}

template <auto kern, typename Params>
cudaError_t launch(const Params& p, const Maps& maps, const Shape& s, int threads, int smem,
                   cudaStream_t st) {
  static std::atomic<uint64_t> done{0}, wide{0};
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), smem, done);
  if (e == cudaSuccess && s.cluster > 8)
    e = allow_wide_cluster(reinterpret_cast<const void*>(kern), wide);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(s.grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)s.cluster;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = s.cluster > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, p, maps);
}

template <typename T>
bool pairs_ok(const ssmq_rows& r) {
  return !r.p || ((reinterpret_cast<uintptr_t>(r.p) % (2 * sizeof(T))) == 0 &&
                  r.batch_stride % 2 == 0 && r.row_stride % 2 == 0);
}

// Tensor map of a (b, L, d) tensor with boxes of one tile; false when TMA does
// not take it (rows off 16-byte boundaries, a broadcast batch, huge sizes).
template <typename T>
bool map_rows(CUtensorMap* map, const ssmq_rows& r, int64_t b, int64_t L, int64_t d, int channels,
              int len) {
  const int64_t rs = (L > 1 ? r.row_stride : (d + 7) / 8 * 8) * (int64_t)sizeof(T);
  const int64_t bs = b > 1 ? r.batch_stride * (int64_t)sizeof(T) : rs * L;
  const int64_t most = (int64_t)1 << 40;
  if ((reinterpret_cast<uintptr_t>(r.p) & 15u) || rs % 16 || bs % 16 || rs <= 0 ||
      bs <= 0 || rs >= most || bs >= most || L >= ((int64_t)1 << 31) - 65536)
    return false;
  const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)L, (cuuint64_t)b};
  const cuuint64_t strides[2] = {(cuuint64_t)rs, (cuuint64_t)bs};
  const cuuint32_t box[3] = {(cuuint32_t)channels, (cuuint32_t)len, 1};
  return encode_tiled(map, sizeof(T) == 4 ? CU_TENSOR_MAP_DATA_TYPE_UINT32
                                          : CU_TENSOR_MAP_DATA_TYPE_UINT16,
                      3, r.p, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_NONE,
                      CU_TENSOR_MAP_L2_PROMOTION_L2_128B) == cudaSuccess;
}

}  // namespace gated
}  // namespace ssmq
