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

template <typename T, bool kVec, int kLanes>
__device__ __forceinline__ Pair<T> load_pair(const T* p, bool in0, bool in1) {
  Pair<T> r;
  if constexpr (kVec) {
    r = Pair<T>{};
    if (in0) r = *reinterpret_cast<const Pair<T>*>(p);
  } else {
    if constexpr (sizeof(T) == 4) {
      r.w.x = in0 ? p[0] : 0.0f;
      r.w.y = in1 ? p[kLanes] : 0.0f;
    } else {
      const uint16_t* u = reinterpret_cast<const uint16_t*>(p);
      const uint32_t a = in0 ? u[0] : 0u, b = in1 ? u[kLanes] : 0u;
      r.w = a | (b << 16);
    }
  }
  return r;
}
template <typename T, bool kVec, int kLanes>
__device__ __forceinline__ void store_pair(T* p, float2 v, bool in0, bool in1) {
  if constexpr (kVec) {
    if (in0) {
      if constexpr (sizeof(T) == 4)
        *reinterpret_cast<float2*>(p) = v;
      else
        *reinterpret_cast<uint32_t*>(p) = pack2<T>(v.x, v.y);
    }
  } else {
    if (in0) p[0] = from_f32<T>(v.x);
    if (in1) p[kLanes] = from_f32<T>(v.y);
  }
}

// f = sigmoid(g), n = 1 - f = sigmoid(-g): the smaller one as e / (1 + e),
// e = exp(-|g|), with full relative accuracy, the larger one as 1 - it.
__device__ __forceinline__ void gate_pair(float g, float& f, float& n) {
  const float e = ex2_sfu(-fabsf(g) * kLog2e);
  const float s = e * rcp_sfu(1.0f + e);
  const float l = 1.0f - s;
  f = g >= 0.0f ? l : s;
  n = g >= 0.0f ? s : l;
}
__device__ __forceinline__ float sigmoid_sfu(float z) {
  return rcp_sfu(1.0f + ex2_sfu(-z * kLog2e));
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
  return make_float2(fmaf(m.x, h.x, m.z), fmaf(m.y, h.y, m.w));
}
// first m, then n
__device__ __forceinline__ float4 compose(float4 m, float4 n) {
  return make_float4(m.x * n.x, m.y * n.y, fmaf(n.x, m.z, n.z), fmaf(n.y, m.w, n.w));
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
  float4 pre = make_float4(1.0f, 1.0f, 0.0f, 0.0f), all = pre;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) {
    if (i == w) pre = all;
    all = compose(all, sh.warp[buf][i][l]);
  }
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
  // Enough CTAs for two per SM, first by splitting time over a cluster, then
  // by narrower channel blocks (32-byte rows of 16-bit elements).
  const int64_t want = 2 * (int64_t)sm_count();
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
  if (n < want) {
    const Shape wide = s;
    s.narrow = true;
    const int64_t m = pick(Tile<8>::kChannels, Tile<8>::kLen);
    if (m <= n || L <= Tile<8>::kLen / 2) s = wide;
    else n = m;
  }
  s.grid = (unsigned)n;
  return s;
}

template <typename Kernel, typename Params>
cudaError_t launch(Kernel kern, const Params& p, const Shape& s, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(s.grid);
  cfg.blockDim = dim3(kThreads);
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
