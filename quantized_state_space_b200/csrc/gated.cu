// Gated linear recurrence, forward and single-token forms (sm_100a).
//
// f_t = sigmoid(g_t), h_t = f_t h_{t-1} + (1 - f_t) v_t, y_t = h_t (silu(z_t)).
// The recurrence is the selective scan's (Quamba2 abstract) with one state per
// channel and the decay as an input.
//
// Bound: HBM (v, g, z in, y out).  The inputs are read once: a tile's gates
// stay in registers while the carried states are exchanged (gated.cuh).  Where a
// tile has two buffers or more (TMA, ungated binary32) the next rounds' rows arrive
// in shared memory meanwhile; with one buffer a round reads its own rows first.
#include "gated.cuh"

namespace ssmq {
namespace {

using namespace gated;

// CTAs per SM that the registers of a mode's kernel are bounded for.
template <typename T, int kMode>
constexpr int kScanCtas = kMode == kTma ? 3 : (sizeof(T) == 4 ? 2 : 3);
// A tile by TMA is fetched into the buffer of the round before the current one;
// what the threads copy takes one buffer (gated binary32: two, which leave room for
// one CTA per SM, took 369 us against 278 at 1 x 12798 x 4394; binary16 pairs: 70
// against 66 at 8 x 2048 x 1538), ungated binary32 two (92 against 98 at
// 52 x 233 x 2717).
template <typename T, int kMode, int kLanes, bool kGate>
using ScanStage = Stage<T, kGate ? 3 : 2, kMode, ModeTile<kMode, kLanes>,
                        kMode == kTma ? (sizeof(T) == 2 && !kGate ? 3 : 2)
                                      : (sizeof(T) == 4 && !kGate ? 2 : 1), true>;

struct ScanParams {
  int64_t L, d, blocks;
  int64_t tiles;        // time tiles of a sequence
  int64_t saved;        // saved states per sequence
  Rows v, g, z, y;
  const float* h0;
  float* h_final;
  float* states;
  const int32_t* lengths;
  uint32_t* status;
  uint32_t wait_limit;  // probes before a wait gives up
};

template <typename T, int kMode, int kLanes, bool kGate>
__global__ void __launch_bounds__(ModeTile<kMode, kLanes>::kThreads, kScanCtas<T, kMode>)
    gated_scan_kernel(const ScanParams p, const __grid_constant__ Maps maps) {
  constexpr bool kVec = kMode != kSingle;
  using TileT = ModeTile<kMode, kLanes>;
  constexpr int kSteps = TileT::kSteps;
  __shared__ Shared<TileT> sh;
  const uint32_t size = cluster_size(), rank = cluster_rank();
  uint32_t live = size, limit = p.wait_limit;  // (see carry_in)
  const int64_t unit = blockIdx.x / size;  // (sequence, channel block)
  const int64_t seq = unit / p.blocks, blk = unit % p.blocks;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = lane / kLanes, l = lane % kLanes;
  using St = ScanStage<T, kMode, kLanes, kGate>;
  constexpr int kNext = St::kNext;
  int64_t c0 = blk * TileT::kChannels + (kNext == 1 ? 2 * l : l);  // first channel
  const bool in0 = c0 < p.d, in1 = c0 + kNext < p.d;
  const int next = in1 ? kNext : 0;
  if (!in0) c0 = 0;
  int64_t end = p.L;
  if (p.lengths) {
    const int64_t n = p.lengths[seq];
    end = n < 0 ? 0 : (n < p.L ? n : p.L);
  }
  const T* vp = static_cast<const T*>(p.v.p) + seq * p.v.bs + c0;
  const T* gp = static_cast<const T*>(p.g.p) + seq * p.g.bs + c0;
  const T* zp = kGate ? static_cast<const T*>(p.z.p) + seq * p.z.bs + c0 : nullptr;
  T* yp = static_cast<T*>(p.y.p) + seq * p.y.bs + c0;
  const int64_t first = (int64_t)(warp * TileT::kSubs + sub) * kSteps;

  float2 h = make_float2(0.0f, 0.0f);
  if (p.h0) h = make_float2(p.h0[seq * p.d + c0], p.h0[seq * p.d + c0 + next]);

  extern __shared__ __align__(128) uint8_t slots[];
  constexpr int kTensors = kGate ? 3 : 2;
  constexpr int kAhead = St::kBufs - 1;  // rounds fetched ahead
  St stage(slots);
  __shared__ uint64_t full[St::kBufs];
  const int64_t rounds = (p.tiles + size - 1) / size;
  uint32_t late = 0;  // a wait gave up
  auto fetch = [&](int64_t k) {
    if (k >= rounds) {
      if constexpr (kMode != kTma) St::commit();
      return;
    }
    const int buf = (int)(k % St::kBufs);
    if constexpr (kMode == kTma) {
      if (threadIdx.x == 0 && !late) {
        const int c = (int)(blk * TileT::kChannels), t = (int)((k * size + rank) * TileT::kLen);
        stream::expect_tx(full + buf, kTensors * St::kTensorBytes);
#pragma unroll
        for (int i = 0; i < kTensors; ++i)
          St::fetch_tile(slots, buf, i, maps.m + i, c, t, (int)seq, full + buf);
      }
    } else {
      const int64_t t0 = (k * size + rank) * TileT::kLen + first;
      const int left = rows_left(end, t0, kSteps);
      stage.fetch(buf, 0, gp + t0 * p.g.rs, p.g.rs, next, left);
      stage.fetch(buf, 1, vp + t0 * p.v.rs, p.v.rs, next, left);
      if constexpr (kGate) stage.fetch(buf, 2, zp + t0 * p.z.rs, p.z.rs, next, left);
      St::commit();
    }
  };
  carry_init(sh, size);
  if constexpr (kMode == kTma) {
    if (threadIdx.x == 0)
      for (int i = 0; i < St::kBufs; ++i) tc::mbar_init(full + i, 1);
    __syncthreads();
  }
  for (int k = 0; k < kAhead; ++k) fetch(k);
  for (int64_t k = 0; k < rounds; ++k) {
    const int buf = (int)(k % St::kBufs);
    if constexpr (kMode == kTma) {
      if (!wait_tile(full + buf, (uint32_t)(k / St::kBufs) & 1u, limit))
        late = 1;
    } else {
      fetch(k + kAhead);
      St::wait();
    }
    const int64_t t0 = (k * size + rank) * TileT::kLen + first;
    float2 f[kSteps], u[kSteps];
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      float2 n;
      gate2(stage.get(buf, 0, i), f[i], n);
      u[i] = fmul2(n, stage.get(buf, 1, i));
    }
    if (end - t0 < kSteps) {  // steps behind the end leave the state
#pragma unroll
      for (int i = 0; i < kSteps; ++i)
        if (i >= end - t0) {
          f[i] = make_float2(1.0f, 1.0f);
          u[i] = make_float2(0.0f, 0.0f);
        }
    }
    float2 a = f[0], b = u[0];
#pragma unroll
    for (int i = 1; i < kSteps; ++i) {
      a = fmul2(a, f[i]);
      b = ffma2(f[i], b, u[i]);
    }
    float2 s = carry_in<TileT, false>(sh, k, make_float4(a.x, a.y, b.x, b.y), h, rank, live,
                                      limit, late, [&] {
                                        // (the tile before this one is read: its buffer is free)
                                        if constexpr (kMode == kTma) fetch(k + kAhead);
                                      });
    if (p.states && t0 < p.L && t0 % kGatedStateSteps == 0) {
      float* o = p.states + (seq * p.saved + t0 / kGatedStateSteps) * p.d + c0;
      if (in0) o[0] = s.x;
      if (in1) o[next] = s.y;
    }
    T* o = yp + t0 * p.y.rs;
    auto put = [&](int i) {
      s = ffma2(f[i], s, u[i]);
      float2 y = s;
      if constexpr (kGate) {
        const float2 z = stage.get(buf, 2, i);
        y = fmul2(s, fmul2(z, sigmoid2(z)));
      }
      return y;
    };
    if (t0 + kSteps <= end) {
#pragma unroll
      for (int i = 0; i < kSteps; ++i)
        store_pair<T, kVec>(o + i * p.y.rs, next, put(i), in0, in1);
    } else {
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        const float2 y = t0 + i < end ? put(i) : make_float2(0.0f, 0.0f);
        if (t0 + i < p.L) store_pair<T, kVec>(o + i * p.y.rs, next, y, in0, in1);
      }
    }
  }
  if (kMode == kTma && late && threadIdx.x == 0) {  // the copies in flight land
    const int64_t k = sh.leave_at;
    for (int64_t j = k; j < rounds && j < k + kAhead; ++j)
      wait_tile(full + j % St::kBufs, (uint32_t)(j / St::kBufs) & 1u, kWaitLimit);
  }
  if (p.h_final && rank == 0 && warp == 0 && sub == 0) {
    float* o = p.h_final + seq * p.d + c0;
    if (in0) o[0] = h.x;
    if (in1) o[next] = h.y;
  }
  flag_status(p.status, late ? SSMQ_DEV_TIMEOUT : 0u);
  carry_done(sh, rounds, late);
}

template <typename T>
cudaError_t scan_type(const ssmq_gated_args& a, cudaStream_t st) {
  // (three CTAs an SM for every type and mode: what 16-bit types by TMA hold)
  const Shape s = shape_for(a.batch, a.seqlen, a.dim, 3 * (int64_t)sm_count(), 1);
  const int len = s.narrow ? kNarrowLen : kWideLen;
  ScanParams p;
  p.L = a.seqlen;
  p.d = a.dim;
  p.blocks = s.blocks;
  p.tiles = (a.seqlen + len - 1) / len;
  p.saved = (a.seqlen + kGatedStateSteps - 1) / kGatedStateSteps;
  p.v = rows_of(a.v);
  p.g = rows_of(a.g);
  p.z = rows_of(a.z);
  p.y = rows_of(a.y);
  p.h0 = a.h0;
  p.h_final = a.h_final;
  p.states = a.states;
  p.lengths = a.lengths;
  p.status = a.status;
  p.wait_limit = stream::wait_limit();
  const bool vec = a.dim % 2 == 0 && pairs_ok<T>(a.v) && pairs_ok<T>(a.g) && pairs_ok<T>(a.z) &&
                   pairs_ok<T>(a.y);
  const bool z = a.z.p != nullptr;
  Maps maps = {};
  const int ch = s.narrow ? kNarrowChannels : kWideChannels;
  auto map = [&](int i, const ssmq_rows& r) {
    return map_rows<T>(maps.m + i, r, a.batch, a.seqlen, a.dim, ch, len);
  };
  const int mode = !vec ? kSingle
                        : (map(0, a.g) && map(1, a.v) && (!z || map(2, a.z)) ? kTma : kPairs);
#define SSMQ_GATED(M, N, Z)                       \
  return launch<gated_scan_kernel<T, M, N, Z>>(p, maps, s, (ModeTile<M, N>::kThreads), \
                                               ScanStage<T, M, N, Z>::kBytes, st)
#define SSMQ_GATED_N(N)                                          \
  switch (mode) {                                                \
    case kTma: if (z) SSMQ_GATED(kTma, N, true); SSMQ_GATED(kTma, N, false);       \
    case kPairs: if (z) SSMQ_GATED(kPairs, N, true); SSMQ_GATED(kPairs, N, false); \
    default: if (z) SSMQ_GATED(kSingle, N, true); SSMQ_GATED(kSingle, N, false);   \
  }
  if (s.narrow) {
    SSMQ_GATED_N(8)
  }
  SSMQ_GATED_N(32)
#undef SSMQ_GATED_N
#undef SSMQ_GATED
}

// ---- one token ----------------------------------------------------------------
// Elementwise: eight channels per thread on 16-byte rows, else one.  Bound: HBM
// (the fp32 state in and out), or the launch itself for a few tokens.
constexpr int kUpdThreads = 128;

struct UpdateParams {
  int64_t b, d, per_row, n;  // n = b * per_row work items
  Rows v, g, z, y;
  float* h;
};

template <typename T, bool kVec>
__global__ void __launch_bounds__(kUpdThreads) gated_update_kernel(const UpdateParams p) {
  const int64_t i = (int64_t)blockIdx.x * kUpdThreads + threadIdx.x;
  if (i >= p.n) return;
  const int64_t r = i / p.per_row, c = (i % p.per_row) * (kVec ? 8 : 1);
  const T* vp = static_cast<const T*>(p.v.p) + r * p.v.bs + c;
  const T* gp = static_cast<const T*>(p.g.p) + r * p.g.bs + c;
  const T* zp = p.z.p ? static_cast<const T*>(p.z.p) + r * p.z.bs + c : nullptr;
  T* yp = static_cast<T*>(p.y.p) + r * p.y.bs + c;
  float* hp = p.h + r * p.d + c;
  constexpr int kN = kVec ? 8 : 1;
  float v[kN], g[kN], z[kN], h[kN];
  if constexpr (kVec) {
    const Raw8<T> a = load8(vp), b = load8(gp);
    const Raw8<float> s = load8(hp);
    if (zp) {
      const Raw8<T> e = load8(zp);
      unpack8<T>(e, z);
    }
    unpack8<T>(a, v);
    unpack8<T>(b, g);
    unpack8<float>(s, h);
  } else {
    v[0] = to_f32(vp[0]);
    g[0] = to_f32(gp[0]);
    h[0] = hp[0];
    if (zp) z[0] = to_f32(zp[0]);
  }
  float y[kN];
#pragma unroll
  for (int j = 0; j < kN; ++j) {
    float2 f, n;  // (the second half of the pair is not used)
    gate2(make_float2(g[j], 0.0f), f, n);
    h[j] = fmaf(f.x, h[j], n.x * v[j]);
    y[j] = zp ? h[j] * (z[j] * sigmoid2(make_float2(z[j], 0.0f)).x) : h[j];
  }
  if constexpr (kVec) {
    store8(hp, pack8<float>(h));
    store8(yp, pack8<T>(y));
  } else {
    hp[0] = h[0];
    yp[0] = from_f32<T>(y[0]);
  }
}

template <typename T>
cudaError_t update_type(const ssmq_gated_args& a, cudaStream_t st) {
  const int e = (int)sizeof(T);
  auto ok = [&](const ssmq_rows& r) { return !r.p || rows16(r.p, r.batch_stride, e); };
  const bool vec = a.dim % 8 == 0 && ok(a.v) && ok(a.g) && ok(a.z) && ok(a.y) &&
                   rows16(a.h_final, 0, 4);
  UpdateParams p;
  p.b = a.batch;
  p.d = a.dim;
  p.per_row = vec ? a.dim / 8 : a.dim;
  p.n = a.batch * p.per_row;
  p.v = rows_of(a.v);
  p.g = rows_of(a.g);
  p.z = rows_of(a.z);
  p.y = rows_of(a.y);
  p.h = a.h_final;
  const unsigned grid = (unsigned)((p.n + kUpdThreads - 1) / kUpdThreads);
  if (vec)
    gated_update_kernel<T, true><<<grid, kUpdThreads, 0, st>>>(p);
  else
    gated_update_kernel<T, false><<<grid, kUpdThreads, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_gated_scan(const ssmq_gated_args& a, cudaStream_t st) {
  switch (a.dtype) {
    case SSMQ_F16: return scan_type<__half>(a, st);
    case SSMQ_BF16: return scan_type<__nv_bfloat16>(a, st);
    default: return scan_type<float>(a, st);
  }
}

cudaError_t launch_gated_update(const ssmq_gated_args& a, cudaStream_t st) {
  switch (a.dtype) {
    case SSMQ_F16: return update_type<__half>(a, st);
    case SSMQ_BF16: return update_type<__nv_bfloat16>(a, st);
    default: return update_type<float>(a, st);
  }
}

}  // namespace ssmq
