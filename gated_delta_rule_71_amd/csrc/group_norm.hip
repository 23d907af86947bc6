// Group norm with an activation, channels last, and its gradient.  A token is a sample,
// its heads the groups.  Per (token, head) row of `group` channels
//     m = mean(x),  r = 1 / sqrt(mean((x - m)^2) + eps),  xh = (x - m) r,
//     n = xh w + b,      y = act(n)  or, with a gate z,  y = n act(z),
// with act SiLU or the identity.  With a = dy act'(n) (no gate) or a = dy act(z),
//     dz = dy n act'(z),  dw = sum_t a xh,  db = sum_t a,
//     c = a w,  dx = r (c - mean(c) - xh mean(c xh)).
// Streams bound by memory traffic: a row sits in the registers of LPR lanes, eight
// channels and 16-byte accesses each, so the mean and the centred sum of squares are two
// passes over registers, not over memory.  36112 tokens of 32 heads of 128, gated, bf16:
// 888 MB in 173 us, 5.1 TB/s, what a large copy reaches; 24 tokens 3.3 us, of 8.1 us that
// the host takes to call it.

#include "common.hpp"
#include "gdr_internal.hpp"

namespace gdr {

namespace {

// p = 1 / (1 + e^-x) and q = 1 - p.  For bf16 rows on the hardware base-2 exponential and
// reciprocal: the argument's rounding makes that |x| 2^-24 of p, far below a bf16 step.  For
// float32 rows from e^-|x|, which cannot overflow, and q by itself, as 1 - p would lose it;
// both within 6 2^-24 of themselves for every x.
template <typename T> struct Sigmoid {
  float p, q;
  __device__ __forceinline__ Sigmoid(float x) {
    p = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-x * 1.4426950408889634f));
    q = 1.0f - p;
  }
};
template <> struct Sigmoid<float> {
  float p, q;
  __device__ __forceinline__ Sigmoid(float x) {
    const float e = expf(-fabsf(x)), near = 1.0f / (1.0f + e), far = e * near;
    p = x < 0.0f ? far : near;
    q = x < 0.0f ? near : far;
  }
};
template <typename T> __device__ __forceinline__ float act(float x, int kind) {
  return kind ? x * Sigmoid<T>(x).p : x;
}
template <typename T> __device__ __forceinline__ float act_slope(float x, int kind) {
  const Sigmoid<T> s(x);
  return kind ? s.p * (1.0f + x * s.q) : 1.0f;
}

__device__ __forceinline__ void put8(uint16_t *p, const float (&y)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = static_cast<uint32_t>(f32_to_bf16(y[2 * i])) |
           (static_cast<uint32_t>(f32_to_bf16(y[2 * i + 1])) << 16);
  *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void put8(float *p, const float (&y)[8]) { store8(p, y); }

template <int LPR>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) x += __shfl_xor(x, o);
  return x;
}

// Mean and reciprocal deviation of a row whose lanes hold VPL vectors of eight channels;
// lanes past the row (live false) hold zeros.  x becomes xh.
template <int LPR, int VPL>
__device__ __forceinline__ float normalise(float (&x)[VPL][8], const bool (&live)[VPL], int group,
                                           float eps) {
  float s = 0.0f;
#pragma unroll
  for (int m = 0; m < VPL; ++m)
#pragma unroll
    for (int e = 0; e < 8; ++e) s += x[m][e];
  const float mean = row_sum<LPR>(s) / group;
  float ss = 0.0f;
#pragma unroll
  for (int m = 0; m < VPL; ++m)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      x[m][e] = live[m] ? x[m][e] - mean : 0.0f;
      ss += x[m][e] * x[m][e];
    }
  const float r = 1.0f / sqrtf(row_sum<LPR>(ss) / group + eps);
#pragma unroll
  for (int m = 0; m < VPL; ++m)
#pragma unroll
    for (int e = 0; e < 8; ++e) x[m][e] *= r;
  return r;
}

template <typename T, int VPL>
__device__ __forceinline__ void load_row(const T *p, const bool (&live)[VPL], int step,
                                         float (&x)[VPL][8]) {
#pragma unroll
  for (int m = 0; m < VPL; ++m) {
    if (live[m]) {
      load8(p + m * step, x[m]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[m][e] = 0.0f;
    }
  }
}

template <typename T, int LPR, int VPL, bool GATE>
__global__ void __launch_bounds__(256) group_norm_kernel(const GroupNormParams p) {
  constexpr int RPB = 256 / LPR, STEP = 8 * LPR;
  const int sub = threadIdx.x % LPR;
  const long row = static_cast<long>(blockIdx.x) * RPB + threadIdx.x / LPR;
  const long r = row < p.rows ? row : p.rows - 1;   // clamped: every lane of a row reduces
  const int head = static_cast<int>(r % p.heads);
  bool live[VPL];
#pragma unroll
  for (int m = 0; m < VPL; ++m) live[m] = 8 * sub + m * STEP < p.group;
  const size_t at = static_cast<size_t>(r) * p.group + 8 * sub;
  float x[VPL][8], z[VPL][8];
  load_row<T, VPL>(static_cast<const T *>(p.x) + at, live, STEP, x);
  if constexpr (GATE) load_row<T, VPL>(static_cast<const T *>(p.z) + at, live, STEP, z);
  normalise<LPR, VPL>(x, live, p.group, p.eps);
  const size_t ch = static_cast<size_t>(head) * p.group + 8 * sub;
#pragma unroll
  for (int m = 0; m < VPL; ++m) {
    if (!live[m] || row >= p.rows) continue;
    float w[8], b[8], y[8];
    load8(p.weight + ch + m * STEP, w);
    if (p.bias) load8(p.bias + ch + m * STEP, b);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float n = p.bias ? fmaf(x[m][e], w[e], b[e]) : x[m][e] * w[e];
      y[e] = GATE ? n * act<T>(z[m][e], p.activation) : act<T>(n, p.activation);
    }
    put8(static_cast<T *>(p.out) + at + m * STEP, y);
  }
}

// Gradient.  A block takes hb heads (consecutive lane groups, so that a token's channels are
// read in one run) and `per_block` tokens, tl of them at a time; each lane keeps the weight
// gradient of its channels in registers over the tokens, the block adds its tl token
// lanes through LDS and writes one row of partial sums, and a second kernel adds the
// blocks' rows in a fixed order.  16384 tokens of 16 heads of 128, gated, bf16: 336 MB in
// 80.4 us a call, 4.2 TB/s; 77 us traced, and 5.4 us for the sums (1024 rows of 16 KB).
template <typename T, int LPR, int VPL, bool GATE>
__global__ void __launch_bounds__(256) group_norm_backward_kernel(const GroupNormParams p) {
  constexpr int RPB = 256 / LPR, STEP = 8 * LPR;
  __shared__ float red[2][RPB][8 * LPR * VPL];
  const int sub = threadIdx.x % LPR, gi = threadIdx.x / LPR;
  const int hb = min(p.heads, RPB), tl = RPB / hb;
  const int head = blockIdx.y * hb + gi % hb, lane_t = gi / hb;
  const bool used = lane_t < tl && head < p.heads;
  bool live[VPL];
#pragma unroll
  for (int m = 0; m < VPL; ++m) live[m] = used && 8 * sub + m * STEP < p.group;
  const size_t channels = static_cast<size_t>(p.heads) * p.group;
  const size_t ch = used ? static_cast<size_t>(head) * p.group + 8 * sub : 0;
  float w[VPL][8], b[VPL][8], dw[VPL][8], db[VPL][8];
  load_row<float, VPL>(p.weight + ch, live, STEP, w);
#pragma unroll
  for (int m = 0; m < VPL; ++m)
#pragma unroll
    for (int e = 0; e < 8; ++e) b[m][e] = dw[m][e] = db[m][e] = 0.0f;
  if (p.bias) load_row<float, VPL>(p.bias + ch, live, STEP, b);

  // the next token's rows are loaded while a token is worked on
  const long t0 = static_cast<long>(blockIdx.x) * p.per_block;
  const long t1 = min(t0 + p.per_block, p.tokens);
  Seg8<T> nx[VPL], ny[VPL], nz[VPL];
  auto fetch = [&](long t) {
    const size_t at = static_cast<size_t>(t) * channels + ch;
#pragma unroll
    for (int m = 0; m < VPL; ++m) {
      if (!live[m]) continue;
      nx[m].load(static_cast<const T *>(p.x) + at + m * STEP);
      ny[m].load(static_cast<const T *>(p.dy) + at + m * STEP);
      if constexpr (GATE) nz[m].load(static_cast<const T *>(p.z) + at + m * STEP);
    }
  };
#pragma unroll
  for (int m = 0; m < VPL; ++m) {
    nx[m].zero();
    ny[m].zero();
    nz[m].zero();
  }
  if (used && t0 + lane_t < t1) fetch(t0 + lane_t);
  for (long t = t0 + lane_t; t < t1 && used; t += tl) {
    const size_t at = static_cast<size_t>(t) * channels + ch;
    float x[VPL][8], z[VPL][8], dy[VPL][8];
#pragma unroll
    for (int m = 0; m < VPL; ++m) {
      nx[m].get(x[m]);
      ny[m].get(dy[m]);
      if constexpr (GATE) nz[m].get(z[m]);
    }
    if (t + tl < t1) fetch(t + tl);
    const float r = normalise<LPR, VPL>(x, live, p.group, p.eps);
    float s = 0.0f, sx = 0.0f;
#pragma unroll
    for (int m = 0; m < VPL; ++m) {
      float dz[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float n = fmaf(x[m][e], w[m][e], b[m][e]);
        float a;
        if constexpr (GATE) {
          a = dy[m][e] * act<T>(z[m][e], p.activation);
          dz[e] = dy[m][e] * n * act_slope<T>(z[m][e], p.activation);
        } else {
          a = dy[m][e] * act_slope<T>(n, p.activation);
        }
        dw[m][e] += a * x[m][e];
        db[m][e] += a;
        dy[m][e] = a * w[m][e];
        s += dy[m][e];
        sx += dy[m][e] * x[m][e];
      }
      if constexpr (GATE)
        if (live[m]) put8(static_cast<T *>(p.dz) + at + m * STEP, dz);
    }
    s = row_sum<LPR>(s) / p.group;
    sx = row_sum<LPR>(sx) / p.group;
#pragma unroll
    for (int m = 0; m < VPL; ++m) {
      if (!live[m]) continue;
      float dx[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) dx[e] = r * (dy[m][e] - s - x[m][e] * sx);
      put8(static_cast<T *>(p.out) + at + m * STEP, dx);
    }
  }

#pragma unroll
  for (int m = 0; m < VPL; ++m)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      red[0][gi][8 * sub + m * STEP + e] = dw[m][e];
      red[1][gi][8 * sub + m * STEP + e] = db[m][e];
    }
  __syncthreads();
  if (lane_t != 0 || !used) return;
  float *dst = p.partial + static_cast<size_t>(blockIdx.x) * 2 * channels + ch;
#pragma unroll
  for (int m = 0; m < VPL; ++m) {
    if (!live[m]) continue;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      float y[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float s = 0.0f;
        for (int l = 0; l < tl; ++l) s += red[q][l * hb + gi][8 * sub + m * STEP + e];
        y[e] = s;
      }
      put8(dst + q * channels + m * STEP, y);
    }
  }
}

// dweight and dbias: the column sums of the blocks' rows (dweight's channels, then
// dbias's).  32 columns per block, 16 bytes per lane, the rows dealt over 32 lanes.
__global__ void __launch_bounds__(256) group_norm_sum_kernel(const float *partial, float *dweight,
                                                             float *dbias, int rows,
                                                             long channels) {
  __shared__ float4 red[32][8];
  const int c = threadIdx.x & 7, l = threadIdx.x >> 3;
  const long ch = static_cast<long>(blockIdx.x) * 32 + 4 * c;
  float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  auto add = [&](const float4 &x) {
    s.x += x.x;
    s.y += x.y;
    s.z += x.z;
    s.w += x.w;
  };
  if (ch < 2 * channels) {
#pragma unroll 8
    for (int r = l; r < rows; r += 32)
      add(*reinterpret_cast<const float4 *>(partial + static_cast<size_t>(r) * 2 * channels + ch));
  }
  red[l][c] = s;
  __syncthreads();
  if (l != 0 || ch >= 2 * channels) return;
#pragma unroll
  for (int m = 1; m < 32; ++m) add(red[m][c]);
  if (ch < channels) *reinterpret_cast<float4 *>(dweight + ch) = s;
  else if (dbias) *reinterpret_cast<float4 *>(dbias + ch - channels) = s;
}

template <typename T, int LPR, int VPL>
hipError_t forward_go(const GroupNormParams &p, hipStream_t s) {
  constexpr int RPB = 256 / LPR;
  const dim3 grid(static_cast<unsigned>((p.rows + RPB - 1) / RPB)), block(256);
  if (p.z)
    hipLaunchKernelGGL((group_norm_kernel<T, LPR, VPL, true>), grid, block, 0, s, p);
  else
    hipLaunchKernelGGL((group_norm_kernel<T, LPR, VPL, false>), grid, block, 0, s, p);
  return hipGetLastError();
}

template <typename T, int LPR, int VPL>
hipError_t backward_go(const GroupNormParams &p, hipStream_t s) {
  constexpr int RPB = 256 / LPR;
  const int hb = p.heads < RPB ? p.heads : RPB;
  const dim3 grid(p.blocks, (p.heads + hb - 1) / hb), block(256);
  if (p.z)
    hipLaunchKernelGGL((group_norm_backward_kernel<T, LPR, VPL, true>), grid, block, 0, s, p);
  else
    hipLaunchKernelGGL((group_norm_backward_kernel<T, LPR, VPL, false>), grid, block, 0, s, p);
  return hipGetLastError();
}

// f with the lanes per row (a power of two, eight channels each) and vectors per lane
template <typename F>
hipError_t by_group(int group, F &&f) {
  using std::integral_constant;
  if (group <= 32) return f(integral_constant<int, 4>(), integral_constant<int, 1>());
  if (group <= 64) return f(integral_constant<int, 8>(), integral_constant<int, 1>());
  if (group <= 128) return f(integral_constant<int, 16>(), integral_constant<int, 1>());
  if (group <= 256) return f(integral_constant<int, 32>(), integral_constant<int, 1>());
  if (group <= 512) return f(integral_constant<int, 64>(), integral_constant<int, 1>());
  return f(integral_constant<int, 64>(), integral_constant<int, 2>());
}

}  // namespace

hipError_t launch_group_norm(const GroupNormParams &p, int f32, hipStream_t stream) {
  if (p.rows == 0) return hipSuccess;
  return by_group(p.group, [&](auto lpr, auto vpl) {
    return f32 ? forward_go<float, lpr(), vpl()>(p, stream)
               : forward_go<uint16_t, lpr(), vpl()>(p, stream);
  });
}

int group_norm_backward_blocks(long tokens, int heads, int group) {
  // One workgroup per compute unit while the tokens last, up to four once each lane still
  // has eight tokens: more would write more partial sums than they hide latency (16384
  // tokens of 16 x 128 bf16 with a gate: 512 workgroups without prefetch 129 us, 1024
  // with it 80 us; 1501 tokens of 5 x 96 float32: 62 workgroups 16.8 us, 256 10.4 us).
  int lpr = 4;
  while (lpr < 64 && 8 * lpr < group) lpr *= 2;
  const int rows = 256 / lpr, hb = heads < rows ? heads : rows;
  const long steps = tokens / (rows / hb);   // of all token lanes of a workgroup
  // a token block's workgroups share those numbers (1024 tokens of 512 x 128 bf16 with a
  // gate, 32 workgroups a block: 193 us and 134 MB of partial sums without, 151 us and 17 MB)
  const long wide = (heads + hb - 1) / hb, least = 256 / wide, most = 1024 / wide;
  const long blocks = steps / 8 > least ? steps / 8 : steps < least ? steps : least;
  return static_cast<int>(blocks < 1 ? 1 : blocks < most ? blocks : most < 1 ? 1 : most);
}

hipError_t launch_group_norm_backward(const GroupNormParams &p, int f32, hipStream_t stream) {
  const hipError_t e = by_group(p.group, [&](auto lpr, auto vpl) {
    return f32 ? backward_go<float, lpr(), vpl()>(p, stream)
               : backward_go<uint16_t, lpr(), vpl()>(p, stream);
  });
  if (e != hipSuccess) return e;
  const long channels = static_cast<long>(p.heads) * p.group;
  hipLaunchKernelGGL(group_norm_sum_kernel, dim3(static_cast<unsigned>((2 * channels + 31) / 32)),
                     dim3(256), 0, stream, p.partial, p.dweight, p.dbias, p.blocks, channels);
  return hipGetLastError();
}

}  // namespace gdr
