// Gradient of the gated linear recurrence (sm_100a).
//
// With f = sigmoid(g), n = 1 - f, h_t = f_t h_{t-1} + n_t v_t, y_t = h_t silu(z_t)
// and l_t the gradient that reaches h_t,
//   l_t = dy_t silu(z_t) + c_{t+1},  c_t = f_t l_t  (c behind the last step: dh_final)
//   dv_t = n_t l_t,  dg_t = f_t n_t (h_{t-1} - v_t) l_t,  dz_t = dy_t h_t silu'(z_t).
// c is a second recurrence, run backwards with the same decays: a segment maps
// the c behind it to the c in front of it as c -> A c + R with the A of its
// forward map.
//
// Bound: HBM (v, g, z, dy in, dv, dg, dz out).  A tile's gates stay in
// registers and its inputs in shared memory (copied one round ahead): the forward
// states inside it are rebuilt from the state that the forward call saved at its
// start (one per 64 steps), so neither h nor the gates cross memory, and only c
// travels between the CTAs of a cluster.
#include "gated.cuh"

namespace ssmq {
namespace {

using namespace gated;

constexpr int kGradCtas = 2;  // per SM
// A round's inputs are read before its exchange: the slot refills behind it.
template <typename T, int kMode, int kLanes, bool kGate>
using GradStage = Stage<T, kGate ? 4 : 3, kMode, ModeTile<kMode, kLanes>, sizeof(T) == 2 ? 2 : 1,
                        sizeof(T) == 2 && kMode == kPairs>;

struct GradParams {
  int64_t L, d, blocks;
  int64_t tiles, saved;
  Rows v, g, z, dy, dv, dg, dz;
  const float* states;
  const float* dh_final;
  float* dh0;
  const int32_t* lengths;
  uint32_t* status;
  uint32_t wait_limit;  // probes before a wait gives up
};

template <typename T, int kMode, int kLanes, bool kGate>
__global__ void __launch_bounds__(ModeTile<kMode, kLanes>::kThreads, kGradCtas)
    gated_scan_grad_kernel(const GradParams p, const __grid_constant__ Maps maps) {
  constexpr bool kVec = kMode != kSingle;
  using TileT = ModeTile<kMode, kLanes>;
  constexpr int kSteps = TileT::kSteps;
  __shared__ Shared<TileT> sh;
  __shared__ float4 s_fwd[2][TileT::kWarps][kLanes];
  const uint32_t size = cluster_size(), rank = cluster_rank();
  uint32_t live = size, limit = p.wait_limit;  // (see carry_in)
  const int64_t unit = blockIdx.x / size;
  const int64_t seq = unit / p.blocks, blk = unit % p.blocks;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = lane / kLanes, l = lane % kLanes;
  using St = GradStage<T, kMode, kLanes, kGate>;
  constexpr int kNext = St::kNext;
  const int64_t block = blk * TileT::kChannels;  // first channel
  int64_t c0 = block + (kNext == 1 ? 2 * l : l);
  const bool in0 = c0 < p.d, in1 = c0 + kNext < p.d;
  const int next = in1 ? kNext : 0;
  if (!in0) c0 = 0;
  int64_t end = p.L;
  if (p.lengths) {
    const int64_t n = p.lengths[seq];
    end = n < 0 ? 0 : (n < p.L ? n : p.L);
  }
  const int64_t cin = St::kWords ? block : c0;  // where the copies of inputs start
  const T* vp = static_cast<const T*>(p.v.p) + seq * p.v.bs + cin;
  const T* gp = static_cast<const T*>(p.g.p) + seq * p.g.bs + cin;
  const T* zp = kGate ? static_cast<const T*>(p.z.p) + seq * p.z.bs + cin : nullptr;
  const T* dyp = static_cast<const T*>(p.dy.p) + seq * p.dy.bs + cin;
  T* dvp = static_cast<T*>(p.dv.p) + seq * p.dv.bs + c0;
  T* dgp = static_cast<T*>(p.dg.p) + seq * p.dg.bs + c0;
  T* dzp = kGate ? static_cast<T*>(p.dz.p) + seq * p.dz.bs + c0 : nullptr;
  const int first = (warp * TileT::kSubs + sub) * kSteps;

  float2 c = make_float2(0.0f, 0.0f);
  if (p.dh_final)
    c = make_float2(p.dh_final[seq * p.d + c0], p.dh_final[seq * p.d + c0 + next]);

  extern __shared__ __align__(128) uint8_t slots[];
  St stage(slots);
  stage.rows_at(0, gp, p.g.rs);
  stage.rows_at(1, vp, p.v.rs);
  stage.rows_at(2, dyp, p.dy.rs);
  if constexpr (kGate) stage.rows_at(3, zp, p.z.rs);
  stage.channels = (int)(p.d - block < TileT::kChannels ? p.d - block : TileT::kChannels);
  __shared__ uint64_t full[St::kBufs];
  const int64_t rounds = (p.tiles + size - 1) / size;
  uint32_t late = 0;  // a wait gave up
  // tiles from the last one backwards; rank 0 holds the latest of a round
  auto tile_of = [&](int64_t k) { return p.tiles - 1 - (k * size + rank); };
  auto fetch = [&](int64_t k) {
    const int64_t tile = tile_of(k);
    const int buf = (int)(k % St::kBufs);
    if constexpr (kMode == kTma) {
      if (threadIdx.x == 0 && !late && k < rounds && tile >= 0) {
        const int c = (int)(blk * TileT::kChannels), t = (int)(tile * TileT::kLen);
        stream::expect_tx(full + buf, (kGate ? 4 : 3) * St::kTensorBytes);
#pragma unroll
        for (int i = 0; i < (kGate ? 4 : 3); ++i)
          St::fetch_tile(slots, buf, i, maps.m + i, c, t, (int)seq, full + buf);
      }
    } else {
      if (k < rounds) {
        const int64_t t0 = tile >= 0 ? tile * TileT::kLen + first : 0;
        const int left = tile >= 0 ? rows_left(end, t0, kSteps) : 0;
        stage.fetch(buf, 0, gp + t0 * p.g.rs, p.g.rs, next, left);
        stage.fetch(buf, 1, vp + t0 * p.v.rs, p.v.rs, next, left);
        stage.fetch(buf, 2, dyp + t0 * p.dy.rs, p.dy.rs, next, left);
        if constexpr (kGate) stage.fetch(buf, 3, zp + t0 * p.z.rs, p.z.rs, next, left);
      }
      St::commit();
    }
  };
  carry_init(sh, size);
  if constexpr (kMode == kTma) {
    if (threadIdx.x == 0)
      for (int i = 0; i < St::kBufs; ++i) tc::mbar_init(full + i, 1);
    __syncthreads();
  }
  for (int k = 0; k < St::kBufs; ++k) fetch(k);
  for (int64_t k = 0; k < rounds; ++k) {
    const int buf = (int)(k % St::kBufs);
    const int64_t tile = tile_of(k);
    const bool real = tile >= 0;
    const int64_t t0 = real ? tile * TileT::kLen + first : 0;
    const int left = real ? rows_left(end, t0, kSteps) : 0;
    float2 hs = make_float2(0.0f, 0.0f);  // state before the tile
    if (real) {
      const float* sp = p.states +
                        (seq * p.saved + tile * (TileT::kLen / kGatedStateSteps)) * p.d + c0;
      hs = make_float2(sp[0], sp[next]);
    }
    if constexpr (kMode == kTma) {
      if (real && !wait_tile(full + buf, (uint32_t)(k / St::kBufs) & 1u, limit))
        late = 1;
      if (left < kSteps) stage.clear(buf, left);
    } else {
      St::wait();
    }

    // Gates and the segment's forward map h -> a h + b.  f = 1, n = 0 behind the end.
    float2 f[kSteps], n[kSteps], q[kSteps];
#pragma unroll
    for (int i = 0; i < kSteps; ++i) gate2(stage.get(buf, 0, i), f[i], n[i]);
    if (left < kSteps) {
#pragma unroll
      for (int i = 0; i < kSteps; ++i)
        if (i >= left) {
          f[i] = make_float2(1.0f, 1.0f);
          n[i] = make_float2(0.0f, 0.0f);
        }
    }
    float2 a = f[0], b = fmul2(n[0], stage.get(buf, 1, 0));
#pragma unroll
    for (int i = 1; i < kSteps; ++i) {
      a = fmul2(a, f[i]);
      b = ffma2(f[i], b, fmul2(n[i], stage.get(buf, 1, i)));
    }
    // Forward state before this segment: the saved state through the CTA's earlier
    // segments.
    {
      float4 m = make_float4(a.x, a.y, b.x, b.y);
      constexpr int kSubs = TileT::kSubs;
#pragma unroll
      for (int o = 1; o < kSubs; o <<= 1) {
        const float4 before = shfl_f4(m, (lane - o * kLanes) & 31);
        if (sub >= o) m = compose(before, m);
      }
      if (sub == kSubs - 1) s_fwd[k & 1][warp][l] = m;
      float4 mine = make_float4(1.0f, 1.0f, 0.0f, 0.0f);
      if constexpr (kSubs > 1) {
        const float4 before = shfl_f4(m, (lane - kLanes) & 31);
        if (sub > 0) mine = before;
      }
      late = __syncthreads_or(late);
      if (late) hs = nan2();  // (dz goes out next)
#pragma unroll
      for (int w = 0; w < TileT::kWarps - 1; ++w) {
        const float4 e = s_fwd[k & 1][w][l];
        if (w < warp) hs = apply(e, hs);
      }
      hs = apply(mine, hs);
    }
    // Forward through the segment.  What the gradients need of it is kept as
    // q_t = f_t (h_{t-1} - v_t) and dh_t = dy_t silu(z_t); dz is written here.
    float2 dh[kSteps];
    T* dzo = kGate ? dzp + t0 * p.dz.rs : nullptr;
    auto walk = [&](int i, bool live, bool row) {
      const float2 v = stage.get(buf, 1, i), one = make_float2(1.0f, 1.0f);
      q[i] = fmul2(f[i], fsub2(hs, v));
      hs = ffma2(f[i], hs, fmul2(n[i], v));
      dh[i] = stage.get(buf, 2, i);
      if constexpr (kGate) {
        const float2 z = stage.get(buf, 3, i), s = sigmoid2(z);
        // silu'(z) = s (1 + z (1 - s))
        float2 dz = fmul2(fmul2(dh[i], hs), fmul2(s, ffma2(z, fsub2(one, s), one)));
        dh[i] = fmul2(dh[i], fmul2(z, s));
        if (!live) dz = make_float2(0.0f, 0.0f);
        if (row) store_pair<T, kVec>(dzo, next, dz, in0, in1);
        dzo += p.dz.rs;
      }
    };
    if (left >= kSteps) {
#pragma unroll
      for (int i = 0; i < kSteps; ++i) walk(i, true, true);
    } else {
#pragma unroll
      for (int i = 0; i < kSteps; ++i) walk(i, i < left, real && t0 + i < p.L);
    }
    // The segment's backward map c -> a c + r, and the c behind the segment.
    float2 r = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int i = kSteps - 1; i >= 0; --i) r = fmul2(f[i], fadd2(dh[i], r));
    r = carry_in<TileT, true>(sh, k, make_float4(a.x, a.y, r.x, r.y), c, rank, live, limit, late,
                              [&] {
                                fetch(k + St::kBufs);  // (every thread has read this tile)
                              });
    T* dvo = dvp + (t0 + kSteps - 1) * p.dv.rs;
    T* dgo = dgp + (t0 + kSteps - 1) * p.dg.rs;
    // gradients of step i, from the last step backwards
    auto put = [&](int i, bool live, bool row) {
      const float2 lam = fadd2(dh[i], r);
      r = fmul2(f[i], lam);
      float2 dv = fmul2(n[i], lam);
      float2 dg = fmul2(dv, q[i]);
      if (!live) dv = dg = make_float2(0.0f, 0.0f);
      if (row) {
        store_pair<T, kVec>(dvo, next, dv, in0, in1);
        store_pair<T, kVec>(dgo, next, dg, in0, in1);
      }
      dvo -= p.dv.rs;
      dgo -= p.dg.rs;
    };
    if (left >= kSteps) {
#pragma unroll
      for (int i = kSteps - 1; i >= 0; --i) put(i, true, true);
    } else if (real) {
#pragma unroll
      for (int i = kSteps - 1; i >= 0; --i) put(i, i < left, t0 + i < p.L);
    }
  }
  if (kMode == kTma && late && threadIdx.x == 0) {  // the copies in flight land
    const int64_t k = sh.leave_at;
    for (int64_t j = k; j < rounds && j < k + St::kBufs && tile_of(j) >= 0; ++j)
      wait_tile(full + j % St::kBufs, (uint32_t)(j / St::kBufs) & 1u, kWaitLimit);
  }
  if (p.dh0 && rank == 0 && warp == 0 && sub == 0) {
    float* o = p.dh0 + seq * p.d + c0;
    if (in0) o[0] = c.x;
    if (in1) o[next] = c.y;
  }
  flag_status(p.status, late ? SSMQ_DEV_TIMEOUT : 0u);
  carry_done(sh, rounds, late);
}

template <typename T>
cudaError_t grad_type(const ssmq_gated_grad_args& a, cudaStream_t st) {
  // (four rounds of CTAs: a CTA's start and end weigh less than an idle SM)
  const Shape s = shape_for(a.batch, a.seqlen, a.dim, kGradCtas * (int64_t)sm_count(), 4);
  const int len = s.narrow ? kNarrowLen : kWideLen;
  GradParams p;
  p.L = a.seqlen;
  p.d = a.dim;
  p.blocks = s.blocks;
  p.tiles = (a.seqlen + len - 1) / len;
  p.saved = (a.seqlen + kGatedStateSteps - 1) / kGatedStateSteps;
  p.v = rows_of(a.v);
  p.g = rows_of(a.g);
  p.z = rows_of(a.z);
  p.dy = rows_of(a.dy);
  p.dv = rows_of(a.dv);
  p.dg = rows_of(a.dg);
  p.dz = rows_of(a.dz);
  p.states = a.states;
  p.dh_final = a.dh_final;
  p.dh0 = a.dh0;
  p.lengths = a.lengths;
  p.status = a.status;
  p.wait_limit = stream::wait_limit();
  const bool z = a.z.p != nullptr;
  const bool vec = a.dim % 2 == 0 && pairs_ok<T>(a.v) && pairs_ok<T>(a.g) && pairs_ok<T>(a.dy) &&
                   pairs_ok<T>(a.dv) && pairs_ok<T>(a.dg) &&
                   (!z || (pairs_ok<T>(a.z) && pairs_ok<T>(a.dz)));
  Maps maps = {};
  const int ch = s.narrow ? kNarrowChannels : kWideChannels;
  auto map = [&](int i, const ssmq_rows& r) {
    return map_rows<T>(maps.m + i, r, a.batch, a.seqlen, a.dim, ch, len);
  };
  const int mode = !vec ? kSingle
                        : (map(0, a.g) && map(1, a.v) && map(2, a.dy) && (!z || map(3, a.z))
                               ? kTma
                               : kPairs);
#define SSMQ_GATED(M, N, Z)                                                                  \
  return launch<gated_scan_grad_kernel<T, M, N, Z>>(p, maps, s, (ModeTile<M, N>::kThreads),  \
                                                    GradStage<T, M, N, Z>::kBytes, st)
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

}  // namespace

cudaError_t launch_gated_scan_backward(const ssmq_gated_grad_args& a, cudaStream_t st) {
  switch (a.dtype) {
    case SSMQ_F16: return grad_type<__half>(a, st);
    case SSMQ_BF16: return grad_type<__nv_bfloat16>(a, st);
    default: return grad_type<float>(a, st);
  }
}

}  // namespace ssmq
