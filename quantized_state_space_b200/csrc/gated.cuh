// Building blocks of the gated recurrence h_t = f_t h_{t-1} + (1 - f_t) v_t:
// the tile of one CTA, its loads, and the exchange of carried states between
// the CTAs of a cluster.
//
// A CTA owns a block of channels and, per round, one tile of consecutive
// steps: kLanes lanes hold two channels each, every thread eight consecutive
// steps of its channels in registers, so a warp holds 32 / kLanes segments
// and the CTA kWarps * 32 / kLanes.  A segment acts on the state entering it
// as h -> A h + B; (A, B) of segments, warps and CTAs compose in step order.
// The CTAs of a cluster hold consecutive tiles and push their (A, B) into
// each other's shared memory; one cluster barrier per round replaces a pass
// over the data or a spin on global memory.
#pragma once

#include "internal.h"
#include "tc.cuh"
#include "vec8.cuh"

namespace ssmq {
namespace gated {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kSteps = 8;        // consecutive steps per thread
constexpr int kMaxCluster = 8;   // CTAs along time (portable cluster size)

template <int kLanes>
struct Tile {
  static constexpr int kChannels = 2 * kLanes;
  static constexpr int kSubs = 32 / kLanes;  // segments per warp
  static constexpr int kLen = kWarps * kSubs * kSteps;
};
static_assert(Tile<32>::kLen % kGatedStateSteps == 0, "saved states at tile starts");
static_assert(kGatedStateSteps % kSteps == 0, "saved states at segment starts");

struct Rows {
  void* p;
  int64_t bs, rs;
};
inline Rows rows_of(const ssmq_rows& r) { return Rows{r.p, r.batch_stride, r.row_stride}; }

// two channels of one row: a pair of consecutive elements (kVec), or elements
// kLanes apart
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

// Elements p[0] and p[next] (kVec: one load of a pair).
template <typename T, bool kVec>
__device__ __forceinline__ Pair<T> load_pair(const T* p, int next) {
  Pair<T> r;
  if constexpr (kVec) {
    r = *reinterpret_cast<const Pair<T>*>(p);
  } else if constexpr (sizeof(T) == 4) {
    r.w = make_float2(p[0], p[next]);
  } else {
    const uint16_t* u = reinterpret_cast<const uint16_t*>(p);
    r.w = (uint32_t)u[0] | ((uint32_t)u[next] << 16);
  }
  return r;
}
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

// Staged inputs.  Every thread copies the pairs of its own steps into slots of
// its own ([buffer][tensor][step][thread], conflict-free) one round ahead and
// reads them back itself: no barrier, and no registers held by loads in flight.
template <typename T, int kTensors>
struct Stage {
  // two buffers of 16-bit elements; binary32 has room for one
  static constexpr int kBufs = sizeof(T) == 4 ? 1 : 2;
  static constexpr int kPerBuf = kTensors * kSteps * kThreads;
  static constexpr int kBytes = kBufs * kPerBuf * (int)sizeof(Pair<T>);
  Pair<T>* mine;
  __device__ __forceinline__ Stage(void* smem)
      : mine(static_cast<Pair<T>*>(smem) + threadIdx.x) {}
  __device__ __forceinline__ Pair<T>* at(int buf, int tensor) const {
    return mine + (kBufs == 1 ? 0 : buf) * kPerBuf + tensor * kSteps * kThreads;
  }
  __device__ __forceinline__ float2 get(int buf, int tensor, int i) const {
    return pair_f32<T>(at(buf, tensor)[i * kThreads]);
  }
  // rows 0 .. left - 1 of the thread's steps, zeros behind them.  Lanes without
  // a channel have their pointers clamped to channel 0.
  template <bool kVec>
  __device__ __forceinline__ void fetch(int buf, int tensor, const T* p, int64_t rs, int next,
                                        int left) const {
    Pair<T>* o = at(buf, tensor);
    if constexpr (kVec) {
      const uint32_t dst = tc::smem_u32(o);
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        const int bytes = i < left ? (int)sizeof(Pair<T>) : 0;
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(
                         dst + i * kThreads * (int)sizeof(Pair<T>)),
                     "l"(p + i * rs), "n"(sizeof(Pair<T>)), "r"(bytes)
                     : "memory");
      }
    } else {
      Pair<T> r[kSteps];
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        r[i] = Pair<T>{};
        if (i < left) r[i] = load_pair<T, kVec>(p + i * rs, next);
      }
#pragma unroll
      for (int i = 0; i < kSteps; ++i) o[i * kThreads] = r[i];
    }
  }
  static __device__ __forceinline__ void commit() {
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  template <int kPending>
  static __device__ __forceinline__ void wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(kPending) : "memory");
  }
};
// rows of the segment at t0 that lie before the end, at most kSteps
__device__ __forceinline__ int rows_left(int64_t end, int64_t t0) {
  const int64_t n = end - t0;
  return n < 0 ? 0 : (n < kSteps ? (int)n : kSteps);
}

// e = exp(-g) with the exponent kept below 2^126, r = 1 / (1 + e): n = 1 - f =
// e r and, for g < 0, f = r have full relative accuracy; for g >= 0, f is
// formed as 1 - n (n <= 1/2: half an ulp), not as the approximate reciprocal,
// whose ulp a long memory would accumulate.
__device__ __forceinline__ void gate2(float2 g, float2& f, float2& n) {
  const float2 x = fmul2(g, make_float2(-kLog2e, -kLog2e));
  const float2 e = make_float2(ex2_sfu(fminf(x.x, 126.0f)), ex2_sfu(fminf(x.y, 126.0f)));
  const float2 one = make_float2(1.0f, 1.0f);
  const float2 d = fadd2(one, e);
  const float2 r = make_float2(rcp_sfu(d.x), rcp_sfu(d.y));
  n = fmul2(e, r);
  const float2 c = fsub2(one, n);
  f.x = g.x < 0.0f ? r.x : c.x;
  f.y = g.y < 0.0f ? r.y : c.y;
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
// 16 bytes into the same shared-memory location of CTA `rank` of the cluster
__device__ __forceinline__ void push_f4(float4* local, uint32_t rank, float4 v) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(tc::smem_u32(local)), "r"(rank));
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(a), "f"(v.x), "f"(v.y),
               "f"(v.z), "f"(v.w)
               : "memory");
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

template <int kLanes>
struct Shared {
  float4 warp[2][kWarps][kLanes];
  float4 cta[2][kMaxCluster][kLanes];
};

// State entering this thread's segment, from the segments' maps in step order
// (kReverse: in reverse step order, the last segment of the warp, warp and
// CTA first), and the state behind the whole round in h.  Every thread of the
// cluster calls it; buf alternates between rounds.
template <int kLanes, bool kReverse>
__device__ __forceinline__ float2 carry_in(Shared<kLanes>& sh, int buf, float4 m, float2& h,
                                           uint32_t rank, uint32_t size) {
  constexpr int kSubs = 32 / kLanes;
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
  __syncthreads();
  float4 pre = make_float4(1.0f, 1.0f, 0.0f, 0.0f);
#pragma unroll 1
  for (int i = 0; i < w; ++i) pre = compose(pre, sh.warp[buf][i][l]);
  float4 all = pre;
#pragma unroll 1
  for (int i = w; i < kWarps; ++i) all = compose(all, sh.warp[buf][i][l]);
  float2 base = h;
  if (size > 1) {
    // warp i tells CTA i of the cluster what this CTA's tile does to a state
    if ((uint32_t)warp < size && sub0 == 0) push_f4(&sh.cta[buf][rank][l], (uint32_t)warp, all);
    cluster_sync();
    float2 s = h;
    for (uint32_t r = 0; r < size; ++r) {
      if (r == rank) base = s;
      s = apply(sh.cta[buf][r][l], s);
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
inline Shape shape_for(int64_t b, int64_t L, int64_t d) {
  Shape s;
  // Enough CTAs for eight per SM, first by splitting time over a cluster, then
  // by narrower channel blocks (32-byte rows of 16-bit elements).
  const int64_t want = 8 * (int64_t)sm_count();
  auto pick = [&](int channels, int len) {
    s.blocks = (d + channels - 1) / channels;
    const int64_t tiles = (L + len - 1) / len;
    s.cluster = 1;
    while (s.cluster < kMaxCluster && s.cluster < tiles && b * s.blocks * s.cluster < want)
      s.cluster *= 2;
    return b * s.blocks * s.cluster;
  };
  s.narrow = false;
  int64_t n = pick(Tile<32>::kChannels, Tile<32>::kLen);
  if (n < want / 4) {
    const Shape wide = s;
    s.narrow = true;
    const int64_t m = pick(Tile<8>::kChannels, Tile<8>::kLen);
    if (m <= n || L <= Tile<8>::kLen / 2) s = wide;
    else n = m;
  }
  s.grid = (unsigned)n;
  return s;
}

template <auto kern, typename Params>
cudaError_t launch(const Params& p, const Shape& s, int smem, cudaStream_t st) {
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), smem, done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(s.grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)s.cluster;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = s.cluster > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

template <typename T>
bool pairs_ok(const ssmq_rows& r) {
  return !r.p || ((reinterpret_cast<uintptr_t>(r.p) % (2 * sizeof(T))) == 0 &&
                  r.batch_stride % 2 == 0 && r.row_stride % 2 == 0);
}

}  // namespace gated
}  // namespace ssmq
