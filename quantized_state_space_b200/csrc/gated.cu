// Gated linear recurrence, forward and single-token forms (sm_100a).
//
// f_t = sigmoid(g_t), h_t = f_t h_{t-1} + (1 - f_t) v_t, y_t = h_t (silu(z_t)).
// The recurrence is the selective scan's (Quamba2 abstract) with one state per
// channel and the decay as an input.
//
// Bound: HBM (v, g, z in, y out).  The inputs are read once: a tile's gates
// stay in registers while the carried states are exchanged (gated.cuh), and
// the next round's rows are copied into shared memory meanwhile.
#include "gated.cuh"

namespace ssmq {
namespace {

using namespace gated;

struct ScanParams {
  int64_t L, d, blocks;
  int64_t tiles;        // time tiles of a sequence
  int64_t saved;        // saved states per sequence
  Rows v, g, z, y;
  const float* h0;
  float* h_final;
  float* states;
  const int32_t* lengths;
};

template <typename T, bool kVec, int kLanes, bool kGate>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 4 ? 3 : 4)
    gated_scan_kernel(const ScanParams p) {
  __shared__ Shared<kLanes> sh;
  using TileT = Tile<kLanes>;
  const uint32_t size = cluster_size(), rank = cluster_rank();
  const int64_t unit = blockIdx.x / size;  // (sequence, channel block)
  const int64_t seq = unit / p.blocks, blk = unit % p.blocks;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = lane / kLanes, l = lane % kLanes;
  int64_t c0 = blk * TileT::kChannels + (kVec ? 2 * l : l);
  const bool in0 = c0 < p.d, in1 = c0 + (kVec ? 1 : kLanes) < p.d;
  const int next = kVec ? 1 : (in1 ? kLanes : 0);
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

  extern __shared__ __align__(16) uint8_t slots[];
  using St = Stage<T, kGate ? 3 : 2>;
  const St stage(slots);
  const int64_t rounds = (p.tiles + size - 1) / size;
  auto fetch = [&](int64_t k) {
    const int64_t t0 = (k * size + rank) * TileT::kLen + first;
    const int left = rows_left(end, t0), buf = (int)(k & 1);
    stage.template fetch<kVec>(buf, 0, gp + t0 * p.g.rs, p.g.rs, next, left);
    stage.template fetch<kVec>(buf, 1, vp + t0 * p.v.rs, p.v.rs, next, left);
    if constexpr (kGate) stage.template fetch<kVec>(buf, 2, zp + t0 * p.z.rs, p.z.rs, next, left);
    St::commit();
  };
  if (St::kBufs == 2 && rounds > 0) fetch(0);
  for (int64_t k = 0; k < rounds; ++k) {
    const int buf = (int)(k & 1);
    if (St::kBufs == 1) {
      fetch(k);
      St::template wait<0>();
    } else if (k + 1 < rounds) {
      fetch(k + 1);
      St::template wait<1>();
    } else {
      St::template wait<0>();
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
    float2 s = carry_in<kLanes, false>(sh, buf, make_float4(a.x, a.y, b.x, b.y), h, rank,
                                       size);
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
  if (p.h_final && rank == 0 && warp == 0 && sub == 0) {
    float* o = p.h_final + seq * p.d + c0;
    if (in0) o[0] = h.x;
    if (in1) o[next] = h.y;
  }
}

template <typename T>
cudaError_t scan_type(const ssmq_gated_args& a, cudaStream_t st) {
  const Shape s = shape_for(a.batch, a.seqlen, a.dim);
  const int len = s.narrow ? Tile<8>::kLen : Tile<32>::kLen;
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
  const bool vec = a.dim % 2 == 0 && pairs_ok<T>(a.v) && pairs_ok<T>(a.g) && pairs_ok<T>(a.z) &&
                   pairs_ok<T>(a.y);
  const bool z = a.z.p != nullptr;
#define SSMQ_GATED(V, N, Z) \
  return launch<gated_scan_kernel<T, V, N, Z>>(p, s, Stage<T, Z ? 3 : 2>::kBytes, st)
  if (vec) {
    if (s.narrow) { if (z) SSMQ_GATED(true, 8, true); SSMQ_GATED(true, 8, false); }
    if (z) SSMQ_GATED(true, 32, true);
    SSMQ_GATED(true, 32, false);
  }
  if (s.narrow) { if (z) SSMQ_GATED(false, 8, true); SSMQ_GATED(false, 8, false); }
  if (z) SSMQ_GATED(false, 32, true);
  SSMQ_GATED(false, 32, false);
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
