// Gated linear recurrence, forward and single-token forms (sm_100a).
//
// f_t = sigmoid(g_t), h_t = f_t h_{t-1} + (1 - f_t) v_t, y_t = h_t (silu(z_t)).
// The recurrence is the selective scan's (Quamba2 abstract) with one state per
// channel and the decay as an input.
//
// Bound: HBM (v, g, z in, y out).  The inputs are read once: a tile's steps
// stay in registers while the carried states are exchanged (gated.cuh), and
// the next round's loads are in flight meanwhile.
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
__global__ void __launch_bounds__(kThreads, 2) gated_scan_kernel(const ScanParams p) {
  __shared__ Shared<kLanes> sh;
  using TileT = Tile<kLanes>;
  const uint32_t size = cluster_size(), rank = cluster_rank();
  const int64_t unit = blockIdx.x / size;  // (sequence, channel block)
  const int64_t seq = unit / p.blocks, blk = unit % p.blocks;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = lane / kLanes, l = lane % kLanes;
  const int64_t c0 = blk * TileT::kChannels + (kVec ? 2 * l : l);
  const bool in0 = c0 < p.d, in1 = c0 + (kVec ? 1 : kLanes) < p.d;
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
  if (p.h0) {
    if (in0) h.x = p.h0[seq * p.d + c0];
    if (in1) h.y = p.h0[seq * p.d + c0 + (kVec ? 1 : kLanes)];
  }

  Pair<T> rv[kSteps], rg[kSteps], rz[kSteps];
  auto fetch = [&](int64_t t0) {
    const T* a = vp + t0 * p.v.rs;
    const T* b = gp + t0 * p.g.rs;
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const bool on = t0 + i < end;
      rg[i] = load_pair<T, kVec, kLanes>(b + i * p.g.rs, on && in0, on && in1);
      rv[i] = load_pair<T, kVec, kLanes>(a + i * p.v.rs, on && in0, on && in1);
    }
  };
  auto fetch_z = [&](int64_t t0) {
    const T* a = zp + t0 * p.z.rs;
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const bool on = t0 + i < end;
      rz[i] = load_pair<T, kVec, kLanes>(a + i * p.z.rs, on && in0, on && in1);
    }
  };

  const int64_t rounds = (p.tiles + size - 1) / size;
  fetch((int64_t)rank * TileT::kLen + first);
  for (int64_t k = 0; k < rounds; ++k) {
    const int64_t t0 = (k * size + rank) * TileT::kLen + first;
    if constexpr (kGate) fetch_z(t0);
    float2 f[kSteps], u[kSteps];
    float4 m = make_float4(1.0f, 1.0f, 0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const float2 g = pair_f32<T>(rg[i]), v = pair_f32<T>(rv[i]);
      float2 n;
      gate_pair(g.x, f[i].x, n.x);
      gate_pair(g.y, f[i].y, n.y);
      u[i] = fmul2(n, v);
      if (t0 + i >= end) {
        f[i] = make_float2(1.0f, 1.0f);
        u[i] = make_float2(0.0f, 0.0f);
      }
      const float2 a = fmul2(make_float2(m.x, m.y), f[i]);
      const float2 b = ffma2(f[i], make_float2(m.z, m.w), u[i]);
      m = make_float4(a.x, a.y, b.x, b.y);
    }
    if (k + 1 < rounds) fetch(t0 + (int64_t)size * TileT::kLen);
    float2 s = carry_in<kLanes, false>(sh, (int)(k & 1), m, h, rank, size);
    if (p.states && t0 < p.L && t0 % kGatedStateSteps == 0) {
      float* o = p.states + (seq * p.saved + t0 / kGatedStateSteps) * p.d + c0;
      if (in0) o[0] = s.x;
      if (in1) o[kVec ? 1 : kLanes] = s.y;
    }
    T* o = yp + t0 * p.y.rs;
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      s = ffma2(f[i], s, u[i]);
      float2 y = s;
      if constexpr (kGate) {
        const float2 z = pair_f32<T>(rz[i]);
        y = fmul2(s, make_float2(z.x * sigmoid_sfu(z.x), z.y * sigmoid_sfu(z.y)));
      }
      if (t0 + i >= end) y = make_float2(0.0f, 0.0f);
      const bool on = t0 + i < p.L;
      store_pair<T, kVec, kLanes>(o + i * p.y.rs, y, on && in0, on && in1);
    }
  }
  if (p.h_final && rank == 0 && warp == 0 && sub == 0) {
    float* o = p.h_final + seq * p.d + c0;
    if (in0) o[0] = h.x;
    if (in1) o[kVec ? 1 : kLanes] = h.y;
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
#define SSMQ_GATED(V, N, Z) return launch(gated_scan_kernel<T, V, N, Z>, p, s, st)
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
    float f, n;
    gate_pair(g[j], f, n);
    h[j] = fmaf(f, h[j], n * v[j]);
    y[j] = zp ? h[j] * (z[j] * sigmoid_sfu(z[j])) : h[j];
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
