// The paged latent cache on sm_100a: rows written into pages, and read back.
//
// A page holds page_size rows. A bf16 row is the 576 values themselves
// (512 latent, 64 rotary). An e4m3 row is 656 bytes:
//   [0, 512)   e4m3 codes of the latent dims
//   [512, 528) four fp32 scales, one for each 128 dims
//   [528, 656) the 64 rotary values in bf16
// value = code * scale with scale = 2^e, the least power of two that is at
// least max|y| / 448 over the 128 dims (1 where all are zero), -100 <= e <= 119.
// With a power of two the division by the scale is exact, and so is the decoded
// value in bf16 (4 significant bits, 448 * 2^119 at most; 256 * 2^120 would be
// infinite): the only rounding is that of y / scale to e4m3 (nearest even, at
// most half a step: 2^-4 |y|, or 2^-10 scale below 2^-6 scale), and a reader may
// form the products of a row in bf16 without a second one. Values above 448 *
// 2^119 = 1.75 * 2^127, in the last binade of bf16, are stored as that.
//
// Both kernels move each byte once with whole-line accesses, one warp a token,
// and are bound by HBM for long runs (read-back of 82K e4m3 rows: 28.6 us a call,
// 26.6 in a graph, 5.6 TB/s of 656 bytes read and 1152 written a row, bf16 rows 31.8;
// 16384 rows appended, in a graph: e4m3 8.5 us, 3.5 TB/s, bf16 8.2, the angles'
// latency among it) and by launch latency at decode sizes (32 rows in a graph: 2.3 us).
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "common.cuh"
#include "kernels.h"

namespace ic {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

template <bool FP8>
__global__ void __launch_bounds__(kThreads) latent_append_kernel(const LatentAppendArgs a) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
  if (t >= a.T) return;
  const int64_t slot = a.slots[t];
  // this lane's latent values (dims 8 lane and 256 + 8 lane, eight each) and its
  // rotary pair, requested before the slot is known
  const uint8_t* src = reinterpret_cast<const uint8_t*>(a.kv) + t * a.kv_stride * 2;
  const uint4 w[2] = {*reinterpret_cast<const uint4*>(src + lane * 16),
                      *reinterpret_cast<const uint4*>(src + 512 + lane * 16)};
  uint32_t rot = *reinterpret_cast<const uint32_t*>(
      src + 1024 + 4 * lane);
  if (slot < 0 || slot >= a.num_slots) {
    if (slot != -1 && lane == 0) record_status(a.status, IC_ERR_BAD_INDEX);
    return;
  }
  const int64_t page = slot / a.page_size;
  const int off = static_cast<int>(slot - page * a.page_size);
  uint8_t* dst = static_cast<uint8_t*>(a.cache) + page * a.page_stride + static_cast<int64_t>(off) * (FP8 ? 656 : 1152);
  uint8_t* rdst = dst + (FP8 ? 528 : 1024);
  if (a.pos) {
    const int64_t p = a.pos[t];
    if (a.half) {
      // dims i and i + 32: lane i (< 16) holds dims 2i, 2i + 1; their partners
      // are in lane i + 16
      const uint32_t other = __shfl_xor_sync(0xffffffffu, rot, 16);
      const int i0 = (lane & 15) * 2;
      float y[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float2 r = rope_cos_sin(p, a.freq[i0 + e], a.mscale, false);
        const float mine = bf16_lane(rot, e), theirs = bf16_lane(other, e);
        y[e] = lane < 16 ? mine * r.x - theirs * r.y : theirs * r.y + mine * r.x;
      }
      rot = pack_bf16x2(y[0], y[1]);
    } else {
      const float2 r = rope_cos_sin(p, a.freq[lane], a.mscale, false);
      const float u = bf16_lane(rot, 0), v = bf16_lane(rot, 1);
      rot = pack_bf16x2(u * r.x - v * r.y, u * r.y + v * r.x);
    }
  }
  *reinterpret_cast<uint32_t*>(rdst + 4 * lane) = rot;
  if constexpr (!FP8) {
    *reinterpret_cast<uint4*>(dst + lane * 16) = w[0];
    *reinterpret_cast<uint4*>(dst + 512 + lane * 16) = w[1];
  } else {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint32_t v[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
      // largest finite |y| of the 128 dims (16 lanes)
      float amax = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float x = fabsf(bf16_lane(v[i >> 1], i & 1));
        if (x < INFINITY) amax = fmaxf(amax, x);
      }
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      // amax = m 2^E with m in [1, 2); 448 = 1.75 2^8: the least e with
      // 2^e >= amax / 448 is E - 8, or E - 7 where m > 1.75 (119 at most: see above)
      int e = 0;
      if (amax > 0.f) {
        const uint32_t bits = __float_as_uint(amax);  // a bf16 subnormal (E = -127 here) ends at e = -100 all the same
        e = static_cast<int>(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
        e = e < -100 ? -100 : e > 119 ? 119 : e;
      }
      const float inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);  // 2^-e, -e in [-119, 100]
      uint32_t c[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float2 p0 = make_float2(bf16_lane(v[2 * i], 0) * inv, bf16_lane(v[2 * i], 1) * inv);
        const float2 p1 = make_float2(bf16_lane(v[2 * i + 1], 0) * inv, bf16_lane(v[2 * i + 1], 1) * inv);
        c[i] = static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(p0, __NV_SATFINITE, __NV_E4M3)) |
               (static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(p1, __NV_SATFINITE, __NV_E4M3)) << 16);
      }
      *reinterpret_cast<uint2*>(dst + k * 256 + lane * 8) = make_uint2(c[0], c[1]);
      if ((lane & 15) == 0)
        *reinterpret_cast<float*>(dst + 512 + (2 * k + (lane >> 4)) * 4) = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
    }
  }
}

// Output row r belongs to sequence b with cu[b] <= r < cu[b + 1]. A warp takes
// kRows consecutive rows; lane j < kRows finds the place of row j, so that the
// lookups of a warp are one chain: the sequence (32 probes a step, or none up to
// 32 sequences), the page, the rows. Against 8 rows a warp in two batches, side by
// side: 82K e4m3 rows 27.4 and 29.0 us, 3 sequences of up to 1021 bf16 rows 4.3 and
// 6.3 us.
constexpr int kRows = 4;

template <bool FP8>
__global__ void __launch_bounds__(kThreads) latent_read_kernel(const LatentReadArgs a) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t r0 = (static_cast<int64_t>(blockIdx.x) * kWarps + warp) * kRows;
  int64_t end = a.cu[a.B];
  // up to 32 sequences: lane b has cu[b], and the lookups need no other read
  const bool few = a.B <= 32;
  const int64_t cu0 = few && lane < a.B ? a.cu[lane] : 0;
  // the last b with cu[b] <= r0 lies in [lo, lo + n)
  int lo = 0, n = few ? 1 : a.B;
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int at = lo + lane * step;
    const bool below = lane * step < n && a.cu[at] <= r0;
    const uint32_t m = __ballot_sync(0xffffffffu, below) | 1u;
    const int last = 31 - __clz(m);
    n = n - last * step < step ? n - last * step : step;
    lo += last * step;
  }
  if (end > a.R) {
    if (blockIdx.x == 0 && threadIdx.x == 0) record_status(a.status, IC_ERR_BAD_INDEX);
    end = a.R;
  }
  if (r0 >= end) return;
  int b = lo;
  int64_t first = 0;  // lane j: the sequence of row j, and its first row
  if (few) {
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      const uint32_t m = __ballot_sync(0xffffffffu, lane < a.B && cu0 <= r0 + j) | 1u;
      if (lane == j) b = 31 - __clz(m);
    }
    first = __shfl_sync(0xffffffffu, cu0, b);
  } else if (lane < kRows) {
    while (b + 1 < a.B && a.cu[b + 1] <= r0 + lane) ++b;
    first = a.cu[b];
  }
  int64_t from = -1;  // lane j: byte offset of row j
  if (lane < kRows && r0 + lane < end) {
    const int64_t p = r0 + lane - first;
    if (p >= 0 && p < static_cast<int64_t>(a.table_width) * a.page_size) {
      const int64_t pi = p / a.page_size;
      const int page = a.table[static_cast<int64_t>(b) * a.table_stride + pi];
      if (page >= 0 && page < a.num_pages)
        from = page * a.page_stride + (p - pi * a.page_size) * (FP8 ? kLatentRowFp8 : kLatentRowBf16);
    }
    if (from < 0) record_status(a.status, IC_ERR_BAD_INDEX);
  }
  const uint8_t* src[kRows];
#pragma unroll
  for (int j = 0; j < kRows; ++j) {
    const int64_t o = __shfl_sync(0xffffffffu, from, j);
    src[j] = o < 0 ? nullptr : static_cast<const uint8_t*>(a.cache) + o;
  }
  if constexpr (!FP8) {
    // 72 words of 16 bytes a row
    uint4 w[kRows][3];
#pragma unroll
    for (int j = 0; j < kRows; ++j)
#pragma unroll
      for (int k = 0; k < 3; ++k) {
        w[j][k] = make_uint4(0, 0, 0, 0);
        if (src[j] && lane + 32 * k < 72) w[j][k] = *reinterpret_cast<const uint4*>(src[j] + (lane + 32 * k) * 16);
      }
#pragma unroll
    for (int j = 0; j < kRows; ++j)
      if (r0 + j < end) {
        uint4* dst = reinterpret_cast<uint4*>(a.out + (r0 + j) * 576);
#pragma unroll
        for (int k = 0; k < 3; ++k)
          if (lane + 32 * k < 72) dst[lane + 32 * k] = w[j][k];
      }
  } else {
    // lane l has dims 8 l and 256 + 8 l, so that each store fills whole lines
    uint2 c[kRows][2];
    uint32_t rot[kRows];
    float s[kRows][2];
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      rot[j] = 0;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        c[j][k] = make_uint2(0, 0);
        s[j][k] = 0.f;
        if (src[j]) {
          c[j][k] = *reinterpret_cast<const uint2*>(src[j] + k * 256 + lane * 8);
          s[j][k] = *reinterpret_cast<const float*>(src[j] + 512 + (2 * k + (lane >> 4)) * 4);
        }
      }
      if (src[j]) rot[j] = *reinterpret_cast<const uint32_t*>(src[j] + 528 + lane * 4);
    }
#pragma unroll
    for (int j = 0; j < kRows; ++j)
      if (r0 + j < end) {
        uint8_t* dst = reinterpret_cast<uint8_t*>(a.out + (r0 + j) * 576);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          uint32_t o[4];
          e4m3x8_to_bf16x8(c[j][k], s[j][k], o);
          *reinterpret_cast<uint4*>(dst + k * 512 + lane * 16) = make_uint4(o[0], o[1], o[2], o[3]);
        }
        *reinterpret_cast<uint32_t*>(dst + 1024 + lane * 4) = rot[j];
      }
  }
}

}  // namespace

cudaError_t launch_latent_append(const LatentAppendArgs& a, bool fp8, cudaStream_t stream) {
  const unsigned grid = static_cast<unsigned>((a.T + kWarps - 1) / kWarps);
  if (fp8)
    latent_append_kernel<true><<<grid, kThreads, 0, stream>>>(a);
  else
    latent_append_kernel<false><<<grid, kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_latent_read(const LatentReadArgs& a, bool fp8, cudaStream_t stream) {
  const int rows = kWarps * kRows;
  const unsigned grid = static_cast<unsigned>((a.R + rows - 1) / rows);
  if (fp8)
    latent_read_kernel<true><<<grid, kThreads, 0, stream>>>(a);
  else
    latent_read_kernel<false><<<grid, kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace ic
