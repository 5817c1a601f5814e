// What the kernels of the latent attention share: the tiles of a share and where
// their rows are, and the softmax and output of a block of query rows.
#pragma once

#include <cuda_bf16.h>

#include "common.cuh"
#include "kernels.h"

namespace ic {

namespace {

constexpr int kT = kLatentTile;
constexpr int kSlab = kT * 128;       // 64 rows x 64 dims, bf16
constexpr int kTile = 9 * kSlab;      // 64 rows of 576 dims: slabs 0-7 latent, 8 rotary
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kMove = 8.f;          // log2 units by which a row's maximum may pass its reference

enum : int { kFirst = 1, kLast = 2, kWhole = 4, kEnd = 8, kClear = 16 };
struct TileInfo {
  int b, pos0, len, flags;
  uint32_t mask[2];  // valid rows of the tile
  int slot;          // partial slot of the piece
  int row0;          // bf16: row of the tile's first position within its page
  int64_t at[4];     // dense: byte offset of each 16 rows (e4m3), or page of each box (bf16; -1: none)
};

// M query rows a CTA. Thread (quadrant, lane) of the softmax has query row
// `row` of the block and part `part` of the columns.
template <int M>
struct Rows {
  static constexpr bool kQStage = M == 32;             // Q passes through a stage into TMEM; else it stays in shared memory
  static constexpr int kStages = M == 32 ? 3 : 2;      // tiles in shared memory
  static constexpr int kClears = kStages + 1;          // bf16: tiles with cleared rows that may wait for their product, and one more
  static constexpr int kParts = 128 / M;               // threads that share a row
  static constexpr int kCols = kT / kParts;            // keys of a thread
  static constexpr int kDims = 256 / kParts;           // output dims of a thread in each half
  static constexpr int kPBufs = M == 32 ? 2 : 1;       // tiles of weights
  static constexpr int kP = M * 128;                   // M rows x 64 weights, bf16
  static constexpr int kQSlab = M * 128;               // M rows x 64 dims of Q, bf16
  // TMEM columns: 2 kDims of O, 2 kCols of S, and for M = 32 288 of Q
  static constexpr uint32_t kOutCol = 0, kSCol = 2 * kDims, kQCol = kSCol + 2 * kCols;
};

IC_DEV int64_t clamp_len(const LatentArgs& a, int64_t n) {
  const int64_t most = static_cast<int64_t>(a.table_width) * a.page_size;
  return n < 0 ? 0 : n > most ? most : n;
}
template <bool SPARSE>
IC_DEV int seq_len(const LatentArgs& a, int b) {
  if (SPARSE) return a.k;
  return static_cast<int>(clamp_len(a, a.lens[b]));
}
IC_DEV int tiles_of(int len) { return (len + kT - 1) / kT; }
// First tile of group g of G (in 32 bits where they hold it: a 64-bit division
// costs a microsecond of the start).
IC_DEV int64_t share_start(int g, int64_t total, int G) {
  if (total < (1 << 22) && G < 512) return static_cast<uint32_t>(g) * static_cast<uint32_t>(total) / static_cast<uint32_t>(G);
  return g * total / G;
}
IC_DEV int eff_groups(int groups, int64_t tiles) {
  return tiles < groups ? static_cast<int>(tiles) : groups;
}

// One warp finds the tiles of its group's share, publishes their descriptors and
// asks L2 for their rows: all of them, or (half >= 0) those of one half of a
// tile, where the other CTA of the pair asks for the rest. unit: rows of an entry
// of TileInfo::at. len0: the length of sequence `lane`, read while the CTA set up.
template <bool FP8, bool SPARSE, int kInfo, class Wait>
IC_DEV void find_tiles(const LatentArgs& a, int64_t len0, int group, int unit, int half, TileInfo* infos, int64_t* places,
                       uint64_t* info_full, uint64_t* info_free, Wait wait) {
  const int lane = threadIdx.x & 31;
  // lane l holds the length of sequence cb + l
  int cb = 0, clen = 0;
  auto load_chunk = [&]() { clen = cb + lane < a.B ? seq_len<SPARSE>(a, cb + lane) : 0; };
  // this group's share of all tiles
  int64_t total = 0;
  if (SPARSE) {
    total = static_cast<int64_t>(a.B) * tiles_of(a.k);
  } else {
    for (cb = 0; cb < a.B; cb += 32) {
      const int64_t n = cb == 0 ? len0 : cb + lane < a.B ? a.lens[cb + lane] : 0;
      if (n != clamp_len(a, n)) record_status(a.status, IC_ERR_BAD_INDEX);
      clen = static_cast<int>(clamp_len(a, n));
      total += tiles_of(clen);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  }
  const int G = eff_groups(a.groups, total);
  const int64_t g0 = group < G ? share_start(group, total, G) : 0;
  int64_t g1 = group < G ? share_start(group + 1, total, G) : 0;
  cb = 0;
  if (SPARSE || a.B > 32) load_chunk();  // (else the chunk is still there)
  int64_t cstart = 0;  // first tile of sequence cb
  int b = 0;            // current sequence, bstart its first tile, bt its tiles
  int64_t bstart = 0;
  int bt = 0, blen = 0;
  if (g0 < g1) {
    while (true) {  // the chunk that holds tile g0
      int incl = tiles_of(clen);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      const int all = __shfl_sync(0xffffffffu, incl, 31);
      if (g0 < cstart + all) {
        const uint32_t past = __ballot_sync(0xffffffffu, g0 < cstart + incl);
        const int l = __ffs(past) - 1;
        b = cb + l;
        blen = __shfl_sync(0xffffffffu, clen, l);
        bt = tiles_of(blen);
        bstart = cstart + __shfl_sync(0xffffffffu, incl, l) - bt;
        break;
      }
      cstart += all;
      cb += 32;
      if (cb >= a.B) {  // (lengths that changed under the call)
        g1 = g0;
        break;
      }
      load_chunk();
    }
  }
  int n = static_cast<int>(g1 - g0);
  bool ok = true;
  int t = 0;
  for (; t < n && ok; ++t) {
    const int64_t gt = g0 + t;
    while (gt >= bstart + bt && b + 1 < a.B) {  // the next sequence with tiles
      bstart += bt;
      ++b;
      if (b >= cb + 32) {
        cb += 32;
        load_chunk();
      }
      blen = __shfl_sync(0xffffffffu, clen, b - cb);
      bt = tiles_of(blen);
    }
    if (gt >= bstart + bt) {  // (lengths that changed under the call)
      n = t;
      break;
    }
    const int pos0 = static_cast<int>(gt - bstart) * kT;
    const bool first = t == 0 || gt == bstart;
    const bool last = t == n - 1 || gt == bstart + bt - 1;
    uint32_t m0 = 0, m1 = 0;
    int64_t s0 = -1, s1 = -1;  // sparse: this lane's two rows
    int64_t src = FP8 ? 0 : -1;  // dense: lane l has the place of the tile's l-th unit
    if constexpr (SPARSE) {
      const int64_t num = static_cast<int64_t>(a.num_pages) * a.page_size;
      auto find = [&](int j, bool ask) -> int64_t {
        if (j >= a.k) return -1;
        const int s = a.slots[static_cast<int64_t>(b) * a.k + j];
        if (s < 0 || s >= num) {
          if (s != -1) record_status(a.status, IC_ERR_BAD_INDEX);
          return -1;
        }
        const int page = s / a.page_size;
        const int64_t at = page * a.page_stride + static_cast<int64_t>(s - page * a.page_size) * kLatentRowFp8;
        if (ask) {
#pragma unroll
          for (int i = 0; i < kLatentRowFp8; i += 128) prefetch_l2(a.cache + at + i);
          prefetch_l2(a.cache + at + kLatentRowFp8 - 16);
        }
        return at;
      };
      s0 = find(pos0 + lane, half != 1);
      s1 = find(pos0 + 32 + lane, half != 0);
      m0 = __ballot_sync(0xffffffffu, s0 >= 0);
      m1 = __ballot_sync(0xffffffffu, s1 >= 0);
    } else {
      const int p = pos0 + lane * unit;
      int rows = 0;  // valid rows of the unit
      int64_t ahead = 0;
      uint32_t ahead_bytes = 0;
      if (lane * unit < kT && p < blen) {
        const int pi = p / a.page_size;
        const int page = a.table[static_cast<int64_t>(b) * a.table_stride + pi];
        if (page >= 0 && page < a.num_pages) {
          rows = blen - p < unit ? blen - p : unit;
          constexpr int kRow = FP8 ? kLatentRowFp8 : kLatentRowBf16;
          const int64_t byte = page * a.page_stride + static_cast<int64_t>(p - pi * a.page_size) * kRow;
          src = FP8 ? byte : page;
          ahead = byte;
          ahead_bytes = static_cast<uint32_t>(rows * kRow);
        } else {
          record_status(a.status, IC_ERR_BAD_INDEX);
        }
      }
      // ask L2 for the units
#pragma unroll 1
      for (int i = 0; i * unit < kT; ++i) {
        const int64_t from = __shfl_sync(0xffffffffu, ahead, i);
        const uint32_t bytes = __shfl_sync(0xffffffffu, ahead_bytes, i);
        if (bytes && half != 1 - i * unit / 32 && elect_one()) bulk_prefetch_l2(a.cache + from, bytes);
        __syncwarp();
      }
      // bit r of the mask: row r is in a valid unit, before the end
      const int rows_of = __shfl_sync(0xffffffffu, rows, lane / unit);
      const int rows_of2 = __shfl_sync(0xffffffffu, rows, (32 + lane) / unit);
      m0 = __ballot_sync(0xffffffffu, lane % unit < rows_of);
      m1 = __ballot_sync(0xffffffffu, (32 + lane) % unit < rows_of2);
    }
    if (!wait(&info_free[t % kInfo], ((t / kInfo) & 1) ^ 1)) {
      ok = false;
      break;
    }
    TileInfo& x = infos[t % kInfo];
    if constexpr (SPARSE) {
      places[(t % kInfo) * kT + lane] = s0;
      places[(t % kInfo) * kT + 32 + lane] = s1;
    } else {
      if (lane < 4) x.at[lane] = src;
    }
    __syncwarp();
    if (lane == 0) {
      x.b = b;
      x.pos0 = pos0;
      x.row0 = SPARSE ? 0 : pos0 % a.page_size;
      x.len = blen;
      x.mask[0] = m0;
      x.mask[1] = m1;
      // only a group's first piece starts at the group's start
      x.slot = 2 * group + (bstart <= g0 ? 0 : 1);
      x.flags = (first ? kFirst : 0) | (last ? kLast : 0) |
                (bstart >= g0 && bstart + bt <= g1 ? kWhole : 0) | ((m0 & m1) != 0xffffffffu ? kClear : 0);
      mbar_arrive(&info_full[t % kInfo]);
    }
    __syncwarp();
  }
  if (ok) ok = wait(&info_free[n % kInfo], ((n / kInfo) & 1) ^ 1);
  if (ok && lane == 0) {
    infos[n % kInfo].flags = kEnd;
    mbar_arrive(&info_full[n % kInfo]);
  }
}

// Four warps: softmax and output of M query rows, the first of them row0 of the
// sequence; `block` is their block of partials. load_q(lanes) brings a piece's Q to
// TMEM (M = 32), p_arrive(t) tells of the weights of tile t, o_arrive() of an
// output that has been read. PAIR: the output columns of a pair of CTAs.
template <int M, bool PAIR, class Wait, class WarpArrive, class GetInfo, class LoadQ, class PArrive, class OArrive>
IC_DEV void softmax_rows(const LatentArgs& a, uint32_t tmem, uint8_t* ps, float* xm, uint64_t* s_full, uint64_t* pv_done,
                         uint64_t* q_free, uint64_t* xch, int row0, int block, Wait wait, WarpArrive warp_arrive,
                         GetInfo get_info, LoadQ load_q, PArrive p_arrive, OArrive o_arrive) {
  using R = Rows<M>;
  constexpr int kCols = R::kCols, kDims = R::kDims;
  constexpr uint32_t kOutCol = R::kOutCol, kSCol = R::kSCol;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int quad = warp & 3;
  // of the columns: kCols of a tile's keys, 2 kDims of the output
  const int part = M == 32 ? quad : quad >> 1;
  const int r = M == 32 ? lane : (quad & 1) * 32 + lane;  // query row of the block
  const uint32_t tlane = tmem + (static_cast<uint32_t>(quad * 32) << 16);
  const float c2 = a.sm_scale * kLog2e;
  const int row = row0 + r;                // query row of the sequence
  const bool live = row < a.rows;
  const int back = a.Q - 1 - (live ? row / a.H : 0);  // the row's token ends this many positions before the last
  const float sink2 = a.sink && live ? a.sink[row % a.H] * kLog2e : -INFINITY;
  float ref = -INFINITY, l = 0.f;
  uint32_t nx = 0;  // exchanges so far
  uint64_t* const xbar = &xch[M == 32 ? 0 : quad & 1];
  auto offer = [&](float v) {
    xm[(nx & 1) * 128 + quad * 32 + lane] = v;
    warp_arrive(xbar);
  };
  auto take = [&](float (&v)[R::kParts]) {  // the values of the row's parts
    const bool ok = wait(xbar, nx & 1);
#pragma unroll
    for (int i = 0; i < R::kParts; ++i) v[i] = xm[(nx & 1) * 128 + (M == 32 ? i : (quad & 1) + 2 * i) * 32 + lane];
    ++nx;
    return ok;
  };
  TileInfo x;
  int pieces = 0;
  bool ok = get_info(0, x);
  if (ok && !(x.flags & kEnd)) ok = load_q(tlane);
  for (int t = 0; ok && !(x.flags & kEnd); ++t) {
    ok = wait(&s_full[t & 1], (t >> 1) & 1);
    if (!ok) break;
    tc_fence_after();
    uint32_t rv[kCols];
    tmem_ld_issue(tlane + kSCol + (t & 1) * kCols, rv);
    if (x.flags & kFirst) {
      ref = -INFINITY;
      l = 0.f;
    }
    constexpr uint32_t kAll = kCols == 32 ? 0xffffffffu : (1u << kCols) - 1;
    uint32_t mask = ((part * kCols & 32 ? x.mask[1] : x.mask[0]) >> (part * kCols & 31)) & kAll;
    const int seen = x.len - back - (x.pos0 + part * kCols);  // columns of this thread before the row's limit
    if (seen < kCols) mask = seen <= 0 ? 0u : mask & ((1u << seen) - 1);
    tmem_ld_wait_for(rv);
    if (!__all_sync(0xffffffffu, mask == kAll)) {
#pragma unroll
      for (int j = 0; j < kCols; ++j)
        if (!((mask >> j) & 1u)) rv[j] = 0xff800000u;  // -inf
    }
    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
    for (int j = 0; j < kCols; ++j) mx[j & 3] = fmaxf(mx[j & 3], __uint_as_float(rv[j]));
    offer(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])));
    // The sum is of the 32-bit weights; those of the product are rounded to bf16
    // (2^-8 of each at most, of either sign), fp32 outputs too: kind::f16 takes
    // both operands in one type, the values are bf16, and a second term of each
    // weight would be as many MMAs again. (The error of bf16 outputs against 64
    // bits is 1.6e-3 to 2.1e-3 of their norm so; their own rounding is 1.65e-3.)
    uint32_t pk[kCols / 2];
    float sum = 0.f;
    auto weigh = [&](float base) {
      float2 part[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
      for (int j = 0; j < kCols; j += 2) {
        const float2 z = ffma2(make_float2(__uint_as_float(rv[j]), __uint_as_float(rv[j + 1])), make_float2(c2, c2),
                              make_float2(-base, -base));
        const float2 w = make_float2(ex2_approx(z.x), ex2_approx(z.y));
        part[(j >> 1) & 1] = add2(part[(j >> 1) & 1], w);
        pk[j >> 1] = pack_bf16x2(w.x, w.y);
      }
      sum = (part[0].x + part[0].y) + (part[1].x + part[1].y);
    };
    // Under the old reference first, which most tiles leave where it is; the
    // other parts' maxima are looked at once everything else has been waited
    // for. (A row with nothing valid so far: every weight is 0.)
    weigh(ref == -INFINITY ? 0.f : ref);
    const TileInfo y = x;
    ok = get_info(t + 1, x);
    if (!ok) break;
    // the product that used this buffer has read its weights
    if (t >= R::kPBufs) ok = wait(&pv_done[(t - R::kPBufs) & 1], ((t - R::kPBufs) >> 1) & 1);
    if (!ok) break;
    float other[R::kParts];
    ok = take(other);
    if (!ok) break;
    float m = other[0];
#pragma unroll
    for (int i = 1; i < R::kParts; ++i) m = fmaxf(m, other[i]);
    m *= c2;
    // the reference moves when the row's maximum passes it by more than kMove:
    // weights stay below 2^8, far from bf16's and fp32's limits
    float scale = 1.f;
    bool moved = false;
    if (ref == -INFINITY) {
      moved = m != -INFINITY;
      ref = m;
    } else if (m > ref + kMove) {
      scale = ex2_approx(ref - m);
      ref = m;
      moved = true;
    }
    if (__any_sync(0xffffffffu, moved)) weigh(ref == -INFINITY ? 0.f : ref);
    l = fmaf(l, scale, sum);
    if (__any_sync(0xffffffffu, scale != 1.f)) {  // (then t > 0, and the warps of a row agree)
      ok = wait(&pv_done[(t - 1) & 1], ((t - 1) >> 1) & 1);  // O stands still
      if (!ok) break;
      tc_fence_after();
#pragma unroll 1
      for (int c = 0; c < 2 * kDims / 32; ++c) {
        uint32_t o[32];
        tmem_ld32_issue(tlane + kOutCol + c * 32, o);
        tmem_ld_wait(o);
#pragma unroll
        for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * scale);
        tmem_st32(tlane + kOutCol + c * 32, o);
      }
      tmem_st_wait();
    }
    const uint32_t pb = smem_u32(ps + (t % R::kPBufs) * R::kP);
#pragma unroll
    for (int i = 0; i < kCols / 8; ++i)
      st_shared_v4(pb + sw128_offset(r, part * (kCols / 8) + i),
                   make_uint4(pk[4 * i], pk[4 * i + 1], pk[4 * i + 2], pk[4 * i + 3]));
    fence_proxy_async_smem();
    tc_fence_before();
    p_arrive(t);
    if (!(y.flags & kLast)) continue;
    // ---- Q of the next piece, and this one's output
    if (M == 32 && !(x.flags & kEnd)) {
      ok = wait(q_free, pieces & 1);
      if (!ok) break;
      tc_fence_after();
      ok = load_q(tlane);
      if (!ok) break;
    }
    ++pieces;
    offer(l);
    float ls[R::kParts];
    ok = take(ls) && wait(&pv_done[t & 1], (t >> 1) & 1);
    if (!ok) break;
    tc_fence_after();
    float lsum = ls[0];
#pragma unroll
    for (int i = 1; i < R::kParts; ++i) lsum += ls[i];
    const bool whole = (y.flags & kWhole) != 0;
    const int64_t gr = (static_cast<int64_t>(y.b) * a.rows) + row;
    const int64_t pb0 = static_cast<int64_t>(y.slot) * a.rblocks + block;  // block of partials
    float f = 1.f;
    if (whole) {
      const float top = fmaxf(ref, sink2);
      const float w = ref == -INFINITY ? 0.f : exp2f(ref - top);
      const float den = lsum * w + (sink2 == -INFINITY ? 0.f : exp2f(sink2 - top));
      f = w > 0.f ? w / den : 0.f;
      if (live && part == 0 && a.lse) a.lse[gr] = top == -INFINITY ? -INFINITY : (top + log2f(den)) / kLog2e;
    } else if (part == 0) {
      reinterpret_cast<float2*>(a.part_ml)[pb0 * M + r] = make_float2(ref, lsum);
    }
#pragma unroll 1
    for (int c = 0; c < 2 * kDims / 32; ++c) {
      uint32_t o[32];
      tmem_ld32_issue(tlane + kOutCol + c * 32, o);
      tmem_ld_wait(o);
      const int dim = PAIR ? part * 256 + c * 32 : c / (kDims / 32) * 256 + part * kDims + c % (kDims / 32) * 32;
      if (!whole) {
        // [block][dim / 4][row][4]: a warp's rows side by side
        uint4* dst = reinterpret_cast<uint4*>(a.part_o) + (pb0 * 128 + dim / 4) * M + r;
#pragma unroll
        for (int k = 0; k < 8; ++k) dst[k * M] = make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
      } else if (live) {
#pragma unroll
        for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
        if (a.gate) {
          const uint4* g = reinterpret_cast<const uint4*>(a.gate + gr * 512 + dim);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint4 w = g[k];
            const uint32_t gw[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int e = 0; e < 8; ++e)
              o[8 * k + e] = __float_as_uint(__uint_as_float(o[8 * k + e]) *
                                             __fdividef(1.f, 1.f + ex2_approx(-kLog2e * bf16_lane(gw[e >> 1], e & 1))));
          }
        }
        if (a.out_f32) {
          uint4* dst = reinterpret_cast<uint4*>(static_cast<float*>(a.out) + gr * 512 + dim);
#pragma unroll
          for (int k = 0; k < 8; ++k) dst[k] = make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
        } else {
          uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + gr * 512 + dim);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              w[e] = pack_bf16x2(__uint_as_float(o[8 * k + 2 * e]), __uint_as_float(o[8 * k + 2 * e + 1]));
            dst[k] = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      }
    }
    tc_fence_before();
    o_arrive();
  }
}

}  // namespace

}  // namespace ic
