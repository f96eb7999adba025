// Residual add + root-mean-square norm + int8 codes with one scale per token
// (sm_100a).
//
// Quamba2 (shd-paper.top card), abstract: W8A8, 8-bit activations in front of
// 8-bit weights.  Per token: r = x + residual rounded to the stream's type,
// rstd = 1 / sqrt(mean r^2 + eps), v = (r w) rstd, scale = max |v| / 127,
// codes = the group quantizer's codes of v at that scale.
//
// Bound: HBM (binary16 with a residual: 7 bytes per element).  A row stays in
// the registers of its threads from the load to the codes, so the row is read
// once.  Because multiplication by rstd > 0 and rounding are monotonic,
// max |fl32((r w) rstd)| = fl32(max |r w| rstd): the sum of squares and the
// maximum are one reduction, with one barrier, instead of two.
#include "internal.h"
#include "quant_fast.cuh"
#include "vec8.cuh"

namespace ssmq {
namespace {

constexpr int kSmallThreads = 128;  // CTA of the rows that fit a warp or less
constexpr int kWideThreads = 512;   // largest CTA that holds one row, to 16384 columns
constexpr int kMaxThreads = 1024;   // and beyond

struct NormParams {
  int64_t tokens;
  int dim;
  float eps, inv_dim;
  const void* x;
  const void* res;
  const float* w;
  void* res_out;
  void* y;
  int8_t* codes;
  float* scales;
  int64_t xs, rs, ros, ys, cs;  // row strides in elements
  uint32_t* status;
};

// codes of eight values at a scale whose reciprocal is usable; false when one
// of them is not finite
__device__ __forceinline__ bool quant8(const float (&v)[8], float s, float rs, uint2& out) {
  const float2 r2 = make_float2(rs, rs), n2 = make_float2(-s, -s);
  const float2 mg = make_float2(12582912.0f, 12582912.0f), zero = make_float2(0.0f, 0.0f);
  float2 nf = zero;
  uint32_t mb[8];
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    float2 q = div2_rn(make_float2(v[i], v[i + 1]), n2, r2);
    nf = ffma2(q, zero, nf);
    q.x = fminf(fmaxf(q.x, -127.0f), 127.0f);
    q.y = fminf(fmaxf(q.y, -127.0f), 127.0f);
    const float2 m = fadd2(q, mg);
    mb[i] = __float_as_uint(m.x);
    mb[i + 1] = __float_as_uint(m.y);
  }
  out.x = __byte_perm(__byte_perm(mb[0], mb[1], 0x0040), __byte_perm(mb[2], mb[3], 0x0040), 0x5410);
  out.y = __byte_perm(__byte_perm(mb[4], mb[5], 0x0040), __byte_perm(mb[6], mb[7], 0x0040), 0x5410);
  return nf.x == 0.0f && nf.y == 0.0f;
}

// How a thread's eight elements of an item lie in the row.
enum {
  kAligned = 0,  // eight consecutive columns, rows on 16-byte boundaries
  kShifted = 1,  // eight consecutive columns on a 16-byte boundary of memory: the
                 // row starts `mis` elements into a piece (the same for every
                 // tensor of 16- or 32-bit elements), its ends go by element
  kScalar = 2    // element e is column e * lanes + lane
};

// kTpr lanes per row (at most a warp), or a CTA size bound: the whole CTA
// holds one row.
template <typename T, int kItems, int kTpr, int kMode>
__global__ void __launch_bounds__(kTpr <= 32 ? kSmallThreads : kTpr)
    rms_norm_quantize_kernel(const NormParams p) {
  __shared__ float s_sum[kMaxThreads / 32], s_max[kMaxThreads / 32];
  constexpr bool kInWarp = kTpr <= 32;
  constexpr bool kPieces = kMode != kScalar;
  const int lanes = kInWarp ? kTpr : (int)blockDim.x;
  const int lane = kInWarp ? (int)threadIdx.x % kTpr : (int)threadIdx.x;
  const int64_t t0 = kInWarp ? (int64_t)blockIdx.x * (kSmallThreads / kTpr) + threadIdx.x / kTpr
                             : (int64_t)blockIdx.x;
  const bool row = t0 < p.tokens;  // (idle rows of the last CTA take part in the shuffles)
  const int64_t t = row ? t0 : 0;
  const T* x = static_cast<const T*>(p.x) + t * p.xs;
  const T* rp = static_cast<const T*>(p.res) + t * p.rs;
  T* ro = static_cast<T*>(p.res_out) + t * p.ros;
  constexpr int kUnit = 16 / (int)sizeof(T);
  const int mis =
      kMode == kShifted ? (int)(reinterpret_cast<uintptr_t>(x) / sizeof(T)) & (kUnit - 1) : 0;
  auto col = [&](int i, int j) -> int {
    return kPieces ? (i * lanes + lane) * 8 + j - mis : (i * 8 + j) * lanes + lane;
  };
  auto inside = [&](int c) { return kMode == kShifted ? c >= 0 && c < p.dim : c < p.dim; };
  auto whole = [&](int c) {  // the piece at column c lies in the row
    return kMode == kShifted ? c >= 0 && c + 8 <= p.dim : c < p.dim;
  };
  // eight elements of a row; 0 outside it
  auto read = [&](const T* q, int i, float (&o)[8]) {
    const int c = col(i, 0);
    if constexpr (kPieces) {
      if (whole(c)) {
        const Raw8<T> r = load8(q + c);
        unpack8<T>(r, o);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          o[j] = kMode == kShifted && inside(c + j) ? to_f32(q[c + j]) : 0.0f;
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = to_f32(q[min(col(i, j), p.dim - 1)]);
    }
  };
  auto write = [&](T* q, int i, const float (&v)[8]) {
    const int c = col(i, 0);
    if constexpr (kPieces) {
      if (whole(c)) {
        store8(q + c, pack8<T>(v));
      } else if (kMode == kShifted) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (inside(c + j)) q[c + j] = from_f32<T>(v[j]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (inside(col(i, j))) q[col(i, j)] = from_f32<T>(v[j]);
    }
  };

  float v[kItems][8];
  float sum = 0.0f, mx = 0.0f;
  if (p.res) {
    float r[kItems][8];
#pragma unroll
    for (int i = 0; i < kItems; ++i) read(x, i, v[i]);
#pragma unroll
    for (int i = 0; i < kItems; ++i) read(rp, i, r[i]);
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] += r[i][j];
      const Raw8<T> o = pack8<T>(v[i]);
      unpack8<T>(o, v[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < kItems; ++i) read(x, i, v[i]);
  }
  if (p.res_out && row) {
#pragma unroll
    for (int i = 0; i < kItems; ++i) write(ro, i, v[i]);
  }

#pragma unroll
  for (int i = 0; i < kItems; ++i) {
    float w[8];
    const int c = col(i, 0);
    if (p.w) {
      if constexpr (kMode == kAligned) {
        if (c < p.dim) {
          const Raw8<float> r = load8(p.w + c);
          unpack8<float>(r, w);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = __ldg(p.w + max(0, min(col(i, j), p.dim - 1)));
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const bool in = inside(col(i, j));
      if (kMode == kScalar && !in) v[i][j] = 0.0f;
      sum = fmaf(v[i][j], v[i][j], sum);
      if (p.w) v[i][j] = in ? v[i][j] * w[j] : 0.0f;
      const float m = fabsf(v[i][j]);
      mx = isfinite(m) ? fmaxf(mx, m) : mx;
    }
  }
#pragma unroll
  for (int o = (kInWarp ? kTpr : 32) / 2; o > 0; o >>= 1) {
    sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
  }
  if constexpr (!kInWarp) {
    const int warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    if ((threadIdx.x & 31) == 0) s_sum[warp] = sum, s_max[warp] = mx;
    __syncthreads();
    const int l = threadIdx.x & 31;
    sum = l < nw ? s_sum[l] : 0.0f;
    mx = l < nw ? s_max[l] : 0.0f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
      mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
    }
  }

  uint32_t flags = 0;
  const bool good = isfinite(sum);
  const float rstd = rsqrtf(fmaf(sum, p.inv_dim, p.eps));
  const float amax = mx * rstd;
  // (eps = 0 and a zero row: 0 * inf; an overflowing maximum has no finite scale)
  const float s = good && isfinite(amax) ? __fdiv_rn(amax, 127.0f) : 0.0f;
  const float rs = s > 0.0f ? __fdiv_rn(1.0f, s) : 0.0f;
  const bool fast = usable_recip(s, rs);
  if (!good) flags |= SSMQ_DEV_NONFINITE;
  if (p.scales && lane == 0 && row) p.scales[t] = s;

  T* y = static_cast<T*>(p.y) + t * p.ys;
  int8_t* q = p.codes + t * p.cs;
#pragma unroll
  for (int i = 0; i < kItems; ++i) {
    const int c = col(i, 0);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[i][j] *= rstd;
    if (p.y && row) write(y, i, v[i]);
    if (!p.codes) continue;
    uint2 out = make_uint2(0u, 0u);
    if (!(s > 0.0f && fast && quant8(v[i], s, rs, out))) {
      uint32_t b[8];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        b[j] = good && inside(col(i, j))
                   ? (uint32_t)quant_elem(v[i][j], s, 0.0f, true, flags) & 0xFFu
                   : 0u;
      out.x = b[0] | (b[1] << 8) | (b[2] << 16) | (b[3] << 24);
      out.y = b[4] | (b[5] << 8) | (b[6] << 16) | (b[7] << 24);
    }
    if constexpr (kMode == kAligned) {
      if (c < p.dim && row) *reinterpret_cast<uint2*>(q + c) = out;
    } else if constexpr (kMode == kShifted) {
      // The piece's codes start `mis` bytes before an 8-byte boundary of the
      // codes' row: the word behind that boundary takes the rest of this piece
      // and the head of the next lane's.  At the ends of a warp (or of the
      // row's lanes), where no lane to the right is at hand, codes go by byte.
      constexpr int kGroup = kInWarp ? kTpr : 32;
      const int g = lane % kGroup;
      const uint64_t own = (uint64_t)out.x | ((uint64_t)out.y << 32);
      const uint64_t right = __shfl_down_sync(0xFFFFFFFFu, own, 1, kGroup);
      const bool edge = mis > 0 && g == kGroup - 1;
      if (row) {
        const int at = c + mis;
        if (!edge && at + 8 <= p.dim) {
          const uint64_t word = mis ? (own >> (8 * mis)) | (right << (64 - 8 * mis)) : own;
          *reinterpret_cast<uint64_t*>(q + at) = word;
        } else {
          const int n = edge ? 8 - mis : 8;
          const uint64_t word =
              mis && !edge ? (own >> (8 * mis)) | (right << (64 - 8 * mis)) : own >> (8 * mis);
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (j < n && at + j < p.dim) q[at + j] = (int8_t)(word >> (8 * j));
        }
        if (g == 0 && mis > 0) {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (j < mis && inside(c + j)) q[c + j] = (int8_t)(own >> (8 * j));
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (row && inside(col(i, j)))
          q[col(i, j)] = (int8_t)((j < 4 ? out.x : out.y) >> (8 * (j & 3)));
    }
  }
  if (row) flag_status(p.status, flags);
}

template <typename T, int kItems, int kTpr, int kMode>
cudaError_t launch_row(const NormParams& p, int lanes, cudaStream_t st) {
  if (kTpr <= 32) {
    const int rows = kSmallThreads / (kTpr <= 32 ? kTpr : 32);
    rms_norm_quantize_kernel<T, kItems, kTpr, kMode>
        <<<(unsigned)((p.tokens + rows - 1) / rows), kSmallThreads, 0, st>>>(p);
  } else {
    rms_norm_quantize_kernel<T, kItems, kTpr, kMode>
        <<<(unsigned)p.tokens, (unsigned)((lanes + 31) / 32 * 32), 0, st>>>(p);
  }
  return cudaGetLastError();
}

// Lanes per row: rows up to 256 elements take one 8-element item per lane,
// wider ones two items per lane, and beyond 2048 four (more loads in flight
// per thread, fewer threads to meet at the barrier).
template <typename T, int kMode>
cudaError_t launch_mode(const NormParams& p, cudaStream_t st) {
  // (a shifted row may touch one piece more than its length says)
  const int pieces = (p.dim + (kMode == kShifted ? 14 : 7)) / 8;
  if (pieces <= 4) return launch_row<T, 1, 4, kMode>(p, 4, st);
  if (pieces <= 8) return launch_row<T, 1, 8, kMode>(p, 8, st);
  if (pieces <= 16) return launch_row<T, 1, 16, kMode>(p, 16, st);
  if (pieces <= 32) return launch_row<T, 1, 32, kMode>(p, 32, st);
  if (pieces <= 64) return launch_row<T, 2, 32, kMode>(p, 32, st);
  if (pieces <= 256) return launch_row<T, 2, kWideThreads, kMode>(p, (pieces + 1) / 2, st);
  if (pieces <= 4 * kWideThreads)
    return launch_row<T, 4, kWideThreads, kMode>(p, (pieces + 3) / 4, st);
  if (pieces <= 4 * kMaxThreads)
    return launch_row<T, 4, kMaxThreads, kMode>(p, (pieces + 3) / 4, st);
  return launch_row<T, 4, kMaxThreads, kScalar>(p, kMaxThreads, st);
}

template <typename T>
cudaError_t launch_type(const NormParams& p, cudaStream_t st) {
  const int e = (int)sizeof(T);
  const bool codes8 = !p.codes || ((reinterpret_cast<uintptr_t>(p.codes) & 7u) == 0 &&
                                   p.cs % 8 == 0);
  if (codes8 && p.dim % 8 == 0 && rows16(p.x, p.xs, e) && (!p.res || rows16(p.res, p.rs, e)) &&
      (!p.res_out || rows16(p.res_out, p.ros, e)) && (!p.y || rows16(p.y, p.ys, e)) &&
      (!p.w || rows16(p.w, 0, 4)))
    return launch_mode<T, kAligned>(p, st);
  // every row of every tensor equally far behind a 16-byte boundary
  auto like_x = [&](const void* q, int64_t stride) {
    return !q || (((reinterpret_cast<uintptr_t>(q) ^ reinterpret_cast<uintptr_t>(p.x)) & 15u) == 0 &&
                  (stride - p.xs) * e % 16 == 0);
  };
  if (codes8 && like_x(p.res, p.rs) && like_x(p.res_out, p.ros) && like_x(p.y, p.ys))
    return launch_mode<T, kShifted>(p, st);
  return launch_mode<T, kScalar>(p, st);
}

}  // namespace

cudaError_t launch_rms_norm_quantize(const ssmq_norm_args& a, cudaStream_t st) {
  NormParams p;
  p.tokens = a.tokens;
  p.dim = (int)a.dim;
  p.eps = a.eps;
  p.inv_dim = 1.0f / (float)a.dim;
  p.x = a.x;
  p.res = a.residual;
  p.w = a.weight;
  p.res_out = a.residual_out;
  p.y = a.y;
  p.codes = a.codes;
  p.scales = a.scales;
  p.xs = a.x_stride;
  p.rs = a.residual_stride;
  p.ros = a.residual_out_stride;
  p.ys = a.y_stride;
  p.cs = a.codes_stride;
  p.status = a.status;
  switch (a.dtype) {
    case SSMQ_F16: return launch_type<__half>(p, st);
    case SSMQ_BF16: return launch_type<__nv_bfloat16>(p, st);
    default: return launch_type<float>(p, st);
  }
}

}  // namespace ssmq
