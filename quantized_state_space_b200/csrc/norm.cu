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
  bool w16;  // w on a 16-byte boundary
};

// Codes of eight values at a scale whose reciprocal is usable; false when one of
// them is not finite.  No clamp: |v| <= max |v| and the scale is fl(max |v| / 127),
// so the quotient is at most 127 (1 + 2^-22) and rounds to 127.
__device__ __forceinline__ bool quant8(const float (&v)[8], float s, float rs, uint2& out) {
  const float2 r2 = make_float2(rs, rs), n2 = make_float2(-s, -s);
  const float2 mg = make_float2(12582912.0f, 12582912.0f), zero = make_float2(0.0f, 0.0f);
  float2 nf = zero;
  uint32_t mb[8];
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    float2 q = div2_rn(make_float2(v[i], v[i + 1]), n2, r2);
    nf = ffma2(q, zero, nf);
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
                 // tensor of 16- or 32-bit elements).  What a piece at an end of
                 // the row writes, and every piece's codes (whose rows start on a
                 // boundary), go through shared memory
  kScalar = 2    // element e is column e * lanes + lane
};

// w[c8 - mis .. c8 - mis + 7] (c8 a multiple of 8, mis < 8) from the four aligned
// 16-byte pieces around them, by three stages of selects: eight loads of single
// weights, 32 bytes apart between lanes, cost four times the cache wavefronts.
// Indices outside the row read some weight of it, or (dim no multiple of 4) the bytes
// behind the last one in its aligned 16: the caller drops both.
__device__ __forceinline__ void shifted_weights(const float* w, int c8, int mis, int dim,
                                                float (&o)[8]) {
  const float4* w4 = reinterpret_cast<const float4*>(w);
  const int last = (dim - 1) / 4;
  float r[16];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float4 q = __ldg(w4 + max(0, min(c8 / 4 - 2 + k, last)));
    r[4 * k] = q.x, r[4 * k + 1] = q.y, r[4 * k + 2] = q.z, r[4 * k + 3] = q.w;
  }
  float a[12], b[9];  // o[j] = r[j + 8 - mis]
#pragma unroll
  for (int i = 0; i < 12; ++i) a[i] = mis & 4 ? r[i] : r[i + 4];
#pragma unroll
  for (int i = 0; i < 9; ++i) b[i] = mis & 2 ? a[i + 1] : a[i + 3];
#pragma unroll
  for (int j = 0; j < 8; ++j) o[j] = mis & 1 ? b[j] : b[j + 1];
}

// kTpr lanes per row (at most a warp), or a CTA size bound: the whole CTA
// holds one row.
template <typename T, int kItems, int kTpr, int kMode>
__global__ void __launch_bounds__(kTpr <= 32 ? kSmallThreads : kTpr)
    rms_norm_quantize_kernel(const NormParams p) {
  __shared__ float s_sum[kMaxThreads / 32], s_max[kMaxThreads / 32];
  constexpr bool kInWarp = kTpr <= 32;
  constexpr bool kPieces = kMode != kScalar;
  constexpr int kRowsCta = kInWarp ? kSmallThreads / (kInWarp ? kTpr : 1) : 1;
  // kShifted: the two end pieces of a row, for residual_out and for y; the codes
  __shared__ __align__(16) T s_ends[kMode == kShifted ? 2 : 1][kMode == kShifted ? kRowsCta : 1][16];
  extern __shared__ __align__(16) uint64_t s_codes[];
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
      } else if (kMode == kShifted && c > -8 && c < p.dim) {
        // an end of the row: the aligned 16 bytes around it, whose other elements
        // (the next row's, padding, or what lies beside the tensor) are dropped; 16
        // bytes without an element of the row are not read
        if constexpr (sizeof(T) == 2) {
          const Raw8<T> r = load8(q + c);
          unpack8<T>(r, o);
        } else {
          const float4 zero = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          const float4* g = reinterpret_cast<const float4*>(q + c);
          unpack8<T>(Raw8<T>{c > -4 ? g[0] : zero, c + 4 < p.dim ? g[1] : zero}, o);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = inside(c + j) ? o[j] : 0.0f;
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = 0.0f;
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = to_f32(q[min(col(i, j), p.dim - 1)]);
    }
  };
  auto meet = [&] {  // the row's threads
    if constexpr (kInWarp)
      __syncwarp();
    else
      __syncthreads();
  };
  const int row_cta = kInWarp ? (int)threadIdx.x / (kInWarp ? kTpr : 1) : 0;
  // kShifted: the row's end pieces from shared memory, an element per lane
  auto write_ends = [&](T* q, int which) {
    const int tail = (p.dim + mis - 1) / 8 * 8 - mis;  // first column of the last piece
    for (int e = lane; e < 16; e += lanes) {
      const int c0 = e < 8 ? -mis : tail, c = c0 + e % 8;
      if (inside(c) && !whole(c0) && (e < 8 || tail > -mis)) q[c] = s_ends[which][row_cta][e];
    }
  };
  auto write = [&](T* q, int i, const float (&v)[8], int which) {
    const int c = col(i, 0);
    if constexpr (kPieces) {
      if (whole(c)) {
        store8(q + c, pack8<T>(v));
      } else if (kMode == kShifted && c > -8 && c < p.dim) {
        store8(&s_ends[kMode == kShifted ? which : 0][row_cta][c <= 0 ? 0 : 8], pack8<T>(v));
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
    for (int i = 0; i < kItems; ++i) write(ro, i, v[i], 0);
  }

  // Sum of squares and the largest |r w|.  Columns outside the row hold 0, and a
  // NaN is passed over by the maximum; an infinity is found afterwards.
#pragma unroll
  for (int i = 0; i < kItems; ++i) {
    float w[8];
    const int c = col(i, 0);
    if (p.w) {
      if (kMode == kAligned && whole(c)) {
        const Raw8<float> r = load8(p.w + c);
        unpack8<float>(r, w);
      } else if (kMode == kShifted && p.w16 && c > -8 && c < p.dim) {
        shifted_weights(p.w, c + mis, mis, p.dim, w);
        if (!whole(c)) {
#pragma unroll
          for (int j = 0; j < 8; ++j) w[j] = inside(c + j) ? w[j] : 0.0f;
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          w[j] = kMode != kAligned && inside(col(i, j)) ? __ldg(p.w + col(i, j)) : 0.0f;
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (kMode == kScalar && !inside(col(i, j))) v[i][j] = 0.0f;
      sum = fmaf(v[i][j], v[i][j], sum);
      if (p.w) v[i][j] *= w[j];
      mx = fmaxf(mx, fabsf(v[i][j]));
    }
  }
  auto reduce = [&](float& add, float& most) {
#pragma unroll
    for (int o = (kInWarp ? kTpr : 32) / 2; o > 0; o >>= 1) {
      add += __shfl_xor_sync(0xFFFFFFFFu, add, o);
      most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, o));
    }
    if constexpr (!kInWarp) {
      const int warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
      if ((threadIdx.x & 31) == 0) s_sum[warp] = add, s_max[warp] = most;
      __syncthreads();
      const int l = threadIdx.x & 31;
      add = l < nw ? s_sum[l] : 0.0f;
      most = l < nw ? s_max[l] : 0.0f;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        add += __shfl_xor_sync(0xFFFFFFFFu, add, o);
        most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, o));
      }
    }
  };
  reduce(sum, mx);
  if constexpr (kMode == kShifted) {
    if (p.res_out) {
      if constexpr (kInWarp) __syncwarp();  // (a CTA's row has met in the reduction)
      if (row) write_ends(ro, 0);
    }
  }
  // an infinite product (in any row of this warp, or in the CTA's row): the maximum
  // over the finite ones
  if (__any_sync(0xFFFFFFFFu, mx > 3.40282347e+38f)) {
    mx = 0.0f;
#pragma unroll
    for (int i = 0; i < kItems; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float m = fabsf(v[i][j]);
        mx = isfinite(m) ? fmaxf(mx, m) : mx;
      }
    if constexpr (!kInWarp) __syncthreads();  // (s_max is read)
    float none = 0.0f;
    reduce(none, mx);
  }

  uint32_t flags = 0;
  const bool good = isfinite(sum);
  const float rstd = rsqrtf(fmaf(sum, p.inv_dim, p.eps));
  float amax = mx * rstd;
  // an infinite value of a finite product (in any row of this warp, or in the CTA's
  // row): the maximum over the finite values
  if (__any_sync(0xFFFFFFFFu, good && amax > 3.40282347e+38f)) {
    amax = 0.0f;
#pragma unroll
    for (int i = 0; i < kItems; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float m = fabsf(v[i][j] * rstd);
        amax = isfinite(m) ? fmaxf(amax, m) : amax;
      }
    if constexpr (!kInWarp) __syncthreads();  // (s_max is read)
    float none = 0.0f;
    reduce(none, amax);
  }
  // (eps = 0 and a zero row: 0 * inf)
  const float s = good && isfinite(amax) ? __fdiv_rn(amax, 127.0f) : 0.0f;
  const float rs = s > 0.0f ? __fdiv_rn(1.0f, s) : 0.0f;
  const bool fast = s > 0.0f && usable_recip(s, rs);
  if (!good) flags |= SSMQ_DEV_NONFINITE;
  if (p.scales && lane == 0 && row) p.scales[t] = s;

  T* y = static_cast<T*>(p.y) + t * p.ys;
  int8_t* q = p.codes + t * p.cs;
#pragma unroll
  for (int i = 0; i < kItems; ++i) {
    const int c = col(i, 0);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[i][j] *= rstd;
    if (p.y && row) write(y, i, v[i], kMode == kShifted ? 1 : 0);
    if (!p.codes) continue;
    uint2 out = make_uint2(0u, 0u);
    if (!(fast && quant8(v[i], s, rs, out))) {
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
      s_codes[(kInWarp ? row_cta * kItems * kTpr : 0) + i * lanes + lane] =
          (uint64_t)out.x | ((uint64_t)out.y << 32);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (row && inside(col(i, j)))
          q[col(i, j)] = (int8_t)((j < 4 ? out.x : out.y) >> (8 * (j & 3)));
    }
  }
  if constexpr (kMode == kShifted) {
    meet();
    if (p.y && row) write_ends(y, 1);
    if (p.codes && row) {
      // aligned words of codes: bytes mis .. of a piece, then the next piece's head
      const uint64_t* from = s_codes + (kInWarp ? row_cta * kItems * kTpr : 0);
#pragma unroll
      for (int i = 0; i < kItems; ++i) {
        const int k = i * lanes + lane;
        if (k * 8 + 8 > p.dim) continue;
        uint64_t word = from[k];
        if (mis) word = (word >> (8 * mis)) | (from[k + 1] << (64 - 8 * mis));
        *reinterpret_cast<uint64_t*>(q + k * 8) = word;
      }
      const int8_t* bytes = reinterpret_cast<const int8_t*>(from);
      for (int c = p.dim / 8 * 8 + lane; c < p.dim; c += lanes) q[c] = bytes[c + mis];
    }
  }
  if (row) flag_status(p.status, flags);
}

template <typename T, int kItems, int kTpr, int kMode>
cudaError_t launch_row(const NormParams& p, int lanes, cudaStream_t st) {
  if (kTpr <= 32) {
    const int rows = kSmallThreads / (kTpr <= 32 ? kTpr : 32);
    rms_norm_quantize_kernel<T, kItems, kTpr, kMode>
        <<<(unsigned)((p.tokens + rows - 1) / rows), kSmallThreads,
           kMode == kShifted ? kSmallThreads * kItems * 8 : 0, st>>>(p);
  } else {
    rms_norm_quantize_kernel<T, kItems, kTpr, kMode>
        <<<(unsigned)p.tokens, (unsigned)((lanes + 31) / 32 * 32),
           kMode == kShifted ? (size_t)((lanes + 31) / 32 * 32) * kItems * 8 : 0, st>>>(p);
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
  p.w16 = (reinterpret_cast<uintptr_t>(a.weight) & 15u) == 0;
  switch (a.dtype) {
    case SSMQ_F16: return launch_type<__half>(p, st);
    case SSMQ_BF16: return launch_type<__nv_bfloat16>(p, st);
    default: return launch_type<float>(p, st);
  }
}

}  // namespace ssmq
