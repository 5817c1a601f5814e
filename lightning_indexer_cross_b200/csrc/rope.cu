// Rotary positions on a [T, H, D] tensor (sm_100a): the rot_dim dims that
// start at rot_off of every head are rotated pairwise by the angle
// position * freq[i], the other dims pass through.
//
//   a = pos[t] * freq[i],  c = mscale cos a,  s = mscale sin a  (transpose: -s)
//   y_u = x_u c - x_v s,   y_v = x_u s + x_v c
//   interleaved: (u, v) = (2i, 2i + 1);  half: (u, v) = (i, i + rot_dim / 2)
//
// The frequency table is 64-bit and the product is reduced modulo 2 pi in
// 64 bits: a 32-bit frequency is off by 2^-24 of itself, 0.06 rad at position
// 10^6. The reduced angle lies in [-pi, pi], where its sine and cosine are
// taken in 32 bits (error below 2^-21), and the rotation is 32-bit, rounded
// once to the tensor's type.
//
// The step reads and writes every element once and computes little: it is
// bound by HBM for long prompts (8192 x 64 x 128, half layout, a call and in a graph:
// bf16 48 and 46 us, 5.8 TB/s, 0.89 of a copy's rate; fp32 88 us in a graph, 6.1
// TB/s) and by launch latency at decode sizes (32 x 128 x 576 bf16: 5.1 and 3.0 us). A CTA
// takes `tpc` tokens x `hpc` heads: its threads first form the tokens' cosines
// and sines in shared memory (once for all heads), then move 16-byte words,
// kUnroll of them in flight a thread.
#include <cuda_bf16.h>

#include "common.cuh"
#include "kernels.h"

namespace ic {

namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;

template <typename T>
struct Vec;
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int N = 8;
  static IC_DEV void unpack(const uint4& w, float (&x)[8]) {
    const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = bf16_lane(a[i >> 1], i & 1);
  }
  static IC_DEV uint4 pack(const float (&x)[8]) {
    return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                      pack_bf16x2(x[6], x[7]));
  }
};
template <>
struct Vec<float> {
  static constexpr int N = 4;
  static IC_DEV void unpack(const uint4& w, float (&x)[4]) {
    x[0] = __uint_as_float(w.x);
    x[1] = __uint_as_float(w.y);
    x[2] = __uint_as_float(w.z);
    x[3] = __uint_as_float(w.w);
  }
  static IC_DEV uint4 pack(const float (&x)[4]) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
  }
};

IC_DEV float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
IC_DEV float to_f(float x) { return x; }
IC_DEV void from_f(__nv_bfloat16& d, float x) { d = __float2bfloat16_rn(x); }
IC_DEV void from_f(float& d, float x) { d = x; }

// Cosines and sines of this CTA's tokens into cs[token][pair].
IC_DEV void fill_table(const RopeArgs& a, float2* cs, int64_t t0, int nt) {
  const int pairs = a.rot_dim / 2;
  for (int i = threadIdx.x; i < nt * pairs; i += kThreads) {
    const int t = i / pairs, p = i - t * pairs;
    cs[i] = rope_cos_sin(a.pos[t0 + t], a.freq[p], a.mscale, a.transpose != 0);
  }
}

// i / d for i d < 2^32, with m = 2^32 / d + 1 from the host: a word's work is
// otherwise half index arithmetic.
struct Div {
  uint32_t d, m;
};
Div make_div(uint32_t d) { return Div{d, d > 1 ? static_cast<uint32_t>((uint64_t(1) << 32) / d + 1) : 0}; }
IC_DEV uint32_t quot(uint32_t i, const Div& v) { return v.d == 1 ? i : __umulhi(i, v.m); }

// 16-byte words. Units of one (token, head) row: `ru` rotated ones (interleaved:
// one word of N / 2 pairs; half: a word of the first half and its partner), and
// `cu` words that are copied (none when the rotation is in place). The first
// rotated words are on their way, and the copies done, before the table is
// needed.
template <typename T, bool HALF>
__global__ void __launch_bounds__(kThreads) rope_vec_kernel(const RopeArgs a, int tpc, int hpc, const Div ru, const Div cu,
                                                            const Div nh_full, const Div nh_last) {
  constexpr int N = Vec<T>::N;
  extern __shared__ __align__(16) float2 cs[];
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * tpc;
  const int nt = a.T - t0 < tpc ? static_cast<int>(a.T - t0) : tpc;
  const int h0 = blockIdx.y * hpc;
  const Div nh = blockIdx.y + 1 == gridDim.y ? nh_last : nh_full;
  const uint32_t rows = nt * nh.d;
  const int pairs = a.rot_dim / 2;
  const T* x = static_cast<const T*>(a.x) + t0 * a.x_ts + h0 * a.x_hs;
  T* y = static_cast<T*>(a.out) + t0 * a.y_ts + h0 * a.y_hs;
  const uint32_t nr = rows * ru.d, nc = rows * cu.d;
  uint4 w0[kUnroll], w1[kUnroll];
  auto load = [&](uint32_t base) {
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) {
      const uint32_t u = base + j * kThreads;
      if (u < nr) {
        const uint32_t row = quot(u, ru), e = u - row * ru.d, t = quot(row, nh), h = row - t * nh.d;
        const T* src = x + t * a.x_ts + h * a.x_hs + a.rot_off + e * N;
        w0[j] = *reinterpret_cast<const uint4*>(src);
        if (HALF) w1[j] = *reinterpret_cast<const uint4*>(src + pairs);
      }
    }
  };
  load(threadIdx.x);
  for (uint32_t base = threadIdx.x; base < nc; base += kThreads * kUnroll) {
    uint4 w[kUnroll];
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) {
      const uint32_t u = base + j * kThreads;
      if (u < nc) {
        const uint32_t row = quot(u, cu), t = quot(row, nh), h = row - t * nh.d;
        int d = (u - row * cu.d) * N;
        if (d >= a.rot_off) d += a.rot_dim;
        w[j] = *reinterpret_cast<const uint4*>(x + t * a.x_ts + h * a.x_hs + d);
      }
    }
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) {
      const uint32_t u = base + j * kThreads;
      if (u < nc) {
        const uint32_t row = quot(u, cu), t = quot(row, nh), h = row - t * nh.d;
        int d = (u - row * cu.d) * N;
        if (d >= a.rot_off) d += a.rot_dim;
        *reinterpret_cast<uint4*>(y + t * a.y_ts + h * a.y_hs + d) = w[j];
      }
    }
  }
  fill_table(a, cs, t0, nt);
  __syncthreads();
  for (uint32_t base = threadIdx.x;;) {
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) {
      const uint32_t u = base + j * kThreads;
      if (u < nr) {
        const uint32_t row = quot(u, ru), e = u - row * ru.d, t = quot(row, nh), h = row - t * nh.d;
        T* dst = y + t * a.y_ts + h * a.y_hs + a.rot_off + e * N;
        const float4* c4 = reinterpret_cast<const float4*>(cs + t * pairs + e * (HALF ? N : N / 2));  // two pairs each
        float p[N];
        Vec<T>::unpack(w0[j], p);
        if constexpr (HALF) {
          float q[N];
          Vec<T>::unpack(w1[j], q);
#pragma unroll
          for (int i = 0; i < N; i += 2) {
            const float4 r = c4[i / 2];
            const float p0 = p[i], q0 = q[i], p1 = p[i + 1], q1 = q[i + 1];
            p[i] = p0 * r.x - q0 * r.y;
            q[i] = p0 * r.y + q0 * r.x;
            p[i + 1] = p1 * r.z - q1 * r.w;
            q[i + 1] = p1 * r.w + q1 * r.z;
          }
          *reinterpret_cast<uint4*>(dst + pairs) = Vec<T>::pack(q);
        } else {
#pragma unroll
          for (int i = 0; i < N / 4; ++i) {
            const float4 r = c4[i];
            const float p0 = p[4 * i], q0 = p[4 * i + 1], p1 = p[4 * i + 2], q1 = p[4 * i + 3];
            p[4 * i] = p0 * r.x - q0 * r.y;
            p[4 * i + 1] = p0 * r.y + q0 * r.x;
            p[4 * i + 2] = p1 * r.z - q1 * r.w;
            p[4 * i + 3] = p1 * r.w + q1 * r.z;
          }
        }
        *reinterpret_cast<uint4*>(dst) = Vec<T>::pack(p);
      }
    }
    base += kThreads * kUnroll;
    if (base >= nr) break;
    load(base);
  }
}

// Any alignment and sizes: one pair, or one copied element, a unit.
template <typename T>
__global__ void __launch_bounds__(kThreads) rope_elem_kernel(const RopeArgs a, int tpc, int hpc, int ru, int cu) {
  extern __shared__ float2 cs[];
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * tpc;
  const int nt = a.T - t0 < tpc ? static_cast<int>(a.T - t0) : tpc;
  const int h0 = blockIdx.y * hpc;
  const int nh = a.H - h0 < hpc ? a.H - h0 : hpc;
  fill_table(a, cs, t0, nt);
  __syncthreads();
  const int upt = nh * (ru + cu);
  const int pairs = a.rot_dim / 2;
  for (int u = threadIdx.x; u < nt * upt; u += kThreads) {
    const int t = u / upt, r = u - t * upt;
    const int h = r / (ru + cu), e = r - h * (ru + cu);
    const T* x = static_cast<const T*>(a.x) + (t0 + t) * a.x_ts + static_cast<int64_t>(h0 + h) * a.x_hs;
    T* y = static_cast<T*>(a.out) + (t0 + t) * a.y_ts + static_cast<int64_t>(h0 + h) * a.y_hs;
    if (e < ru) {
      const int d0 = a.rot_off + (a.half ? e : 2 * e), d1 = d0 + (a.half ? pairs : 1);
      const float2 r2 = cs[t * pairs + e];
      const float p = to_f(x[d0]), q = to_f(x[d1]);
      from_f(y[d0], p * r2.x - q * r2.y);
      from_f(y[d1], p * r2.y + q * r2.x);
    } else {
      int d = e - ru;
      if (d >= a.rot_off) d += a.rot_dim;
      y[d] = x[d];
    }
  }
}

template <typename T>
cudaError_t launch_t(const RopeArgs& a, bool vec, cudaStream_t stream) {
  const int N = Vec<T>::N;
  const bool copy = a.out != a.x || a.x_ts != a.y_ts || a.x_hs != a.y_hs;
  const int ru = vec ? (a.half ? a.rot_dim / 2 / N : a.rot_dim / N) : a.rot_dim / 2;
  const int cu = !copy ? 0 : (a.D - a.rot_dim) / (vec ? N : 1);
  const int per_head = ru + cu;
  // heads per CTA: about kUnroll units a thread; then tokens until the same
  // amount (few heads), bounded by the table
  const int want = kThreads * kUnroll;
  int hpc = (want + per_head - 1) / per_head;
  if (hpc > a.H) hpc = a.H;
  int tpc = want / (hpc * per_head);
  const int most = 4096 / (a.rot_dim / 2);  // 32 KB of table
  if (tpc > most) tpc = most;
  // few tokens: one a CTA, so that their loads spread over the SMs; many: up to
  // four times the work, so that the table's latency (a 64-bit product and a
  // sine) is paid less often (8192 x 64 x 128: 48 us, 64 us without), while eight
  // CTAs an SM remain
  while (tpc > 1 && (a.T + tpc - 1) / tpc < 296) tpc /= 2;
  if (tpc < 1) tpc = 1;
  const int heads = (a.H + hpc - 1) / hpc;
  for (int i = 0; i < 2 && 2 * tpc <= most && (a.T + 2 * tpc - 1) / (2 * tpc) * heads >= 1184; ++i) tpc *= 2;
  if (tpc < 1) tpc = 1;
  const int64_t gx = (a.T + tpc - 1) / tpc;
  const dim3 grid(static_cast<unsigned>(gx), static_cast<unsigned>((a.H + hpc - 1) / hpc));
  const size_t smem = static_cast<size_t>(tpc) * (a.rot_dim / 2) * sizeof(float2);
  if (!vec) {
    rope_elem_kernel<T><<<grid, kThreads, smem, stream>>>(a, tpc, hpc, ru, cu);
    return cudaGetLastError();
  }
  const Div dr = make_div(ru), dc = make_div(cu > 0 ? cu : 1), nf = make_div(hpc), nl = make_div(a.H - (grid.y - 1) * hpc);
  const Div copies{cu > 0 ? dc.d : 0, dc.m};
  if (a.half)
    rope_vec_kernel<T, true><<<grid, kThreads, smem, stream>>>(a, tpc, hpc, dr, copies, nf, nl);
  else
    rope_vec_kernel<T, false><<<grid, kThreads, smem, stream>>>(a, tpc, hpc, dr, copies, nf, nl);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, bool f32, cudaStream_t stream) {
  const int N = f32 ? 4 : 8;
  const int part = a.half ? a.rot_dim / 2 : a.rot_dim;
  const bool vec = ((reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.out)) & 15) == 0 &&
                   a.x_ts % N == 0 && a.x_hs % N == 0 && a.y_ts % N == 0 && a.y_hs % N == 0 && a.D % N == 0 &&
                   a.rot_off % N == 0 && part % N == 0;
  return f32 ? launch_t<float>(a, vec, stream) : launch_t<__nv_bfloat16>(a, vec, stream);
}

}  // namespace ic
