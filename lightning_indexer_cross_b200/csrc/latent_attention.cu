// Latent attention over the paged cache on sm_100a: each of a sequence's
// query rows (Q tokens x H heads, absorbed form) attends to the cached rows,
// whose 576 dims are the keys and whose first 512 dims are the values.
//
//   z_j = sm_scale q . row_j,  o = sum_j e^{z_j} row_j[:512] / (e^{sink} + sum_j e^{z_j})
//   out = sigmoid(gate) o,     lse = log(e^{sink} + sum_j e^{z_j})
//
// Dense: j runs over the positions before the query token's limit, found in
// the pages of the sequence's block table. Sparse: j runs over the given slots
// of the cache.
//
// Split. The tiles of 64 keys of all sequences, one after another, are shared
// out evenly: group g takes tiles [g T / G, (g + 1) T / G), so ragged lengths
// load every SM alike and a single long sequence uses all of them. The lengths
// are read on the device; nothing waits for the host. A group has one CTA for
// each block of 64 query rows; the CTAs of a group read the same tiles at the
// same time, so the second read of a tile hits L2. A piece is what one group
// has of one sequence: whole sequences are finished by their CTA, the others
// leave (reference, sum, unnormalised output) in fp32 and a second kernel
// joins them.
//
// CTA. M = 64 query rows in the weight-stationary MMA form, whose 64 x 512
// output takes 256 of the 512 TMEM columns (the ordinary M = 128 form would
// need all of them and leave none for the logits). Per tile
//   S[64 x 64]   = Q . K^T         (36 MMAs, N = 64)
//   P            = 2^(S sm_scale log2e - ref), bf16 into shared memory
//   O[64 x 512] += P . V           (8 MMAs, N = 256; V is the same tile read
//                                   as an MN-major operand)
// with the running reference of an online softmax, moved (and O rescaled) only
// when a row's maximum passes it by more than 2^8.
//
// Roles. Warp 0 finds the tiles and issues their copies, warp 1 the MMAs, warp
// 2 loads Q, warps 4-7 run the softmax and the output. bf16 pages: TMA boxes
// land in the operand layout; warp 3 clears the rows behind a sequence's end
// (a zero weight times a NaN left there would be NaN). e4m3 pages: rows land
// as they are stored and warps 8-15 widen them into the operand layout.
#include <cuda_bf16.h>

#include "common.cuh"
#include "kernels.h"

namespace ic {

namespace {

constexpr int kT = kLatentTile;
constexpr int kSlab = kT * 128;       // 64 rows x 64 dims, bf16
constexpr int kHalf = 4 * kSlab;      // 64 rows x 256 dims
constexpr int kRawRows = 32;          // rows of an e4m3 staging chunk
constexpr int kRawBytes = kRawRows * kLatentRowFp8;
constexpr int kInfo = 8;              // tile descriptors in flight
constexpr int kMinTiles = 2;          // tiles of a group, at least
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kMove = 8.f;          // log2 units by which a row's maximum may pass its reference

enum : int { kFirst = 1, kLast = 2, kWhole = 4, kEnd = 8, kClear = 16 };
struct TileInfo {
  int b, pos0, len, flags;
  uint32_t mask[2];  // valid rows of the tile
  int slot;          // partial slot of the piece
  int pad;
};

template <bool FP8>
struct Cfg {
  static constexpr int kThreads = FP8 ? 512 : 256;
  static constexpr int kHalves = FP8 ? 2 : 4;  // 32 KB operand slots (latent halves of a tile)
  static constexpr int kRopes = 2;             // 8 KB operand slots (rotary slab of a tile)
  static constexpr int kRaws = FP8 ? 3 : 1;             // e4m3 staging chunks (bf16: none used)
  // QK of a tile is issued before PV of the previous one; needs two tiles of operand slots
  static constexpr int kLag = FP8 ? 0 : 1;
  static constexpr int kOffQ = 0;
  static constexpr int kOffHalf = 9 * kSlab;
  static constexpr int kOffRope = kOffHalf + kHalves * kHalf;
  static constexpr int kOffP = kOffRope + kRopes * kSlab;
  static constexpr int kOffRaw = kOffP + kSlab;
  static constexpr int kOffX = kOffRaw + (FP8 ? kRaws * kRawBytes : 0);  // [2][128] row maxima / sums
  static constexpr int kOffInfo = kOffX + 2 * 128 * 4;
  static constexpr int kOffBar = kOffInfo + kInfo * static_cast<int>(sizeof(TileInfo));
  // readers of a tile descriptor: MMA, Q, four softmax warps, the clearing warp or the widening warps
  static constexpr int kReaders = 6 + (FP8 ? 8 : 1);
  static constexpr int kNumBars = 2 * kInfo + 2 * kHalves + 2 * kRopes + 2 * kRaws + 10;
  static constexpr int kOffMisc = kOffBar + kNumBars * 8;
  static constexpr int kSmemBytes = kOffMisc + 16;
  static_assert(kOffBar % 8 == 0 && kOffRaw % 128 == 0, "alignment");
  static_assert(kSmemBytes <= 232448, "fits one CTA per SM");
  static_assert(kLag == 0 || (kHalves >= 4 && kRopes >= 2), "slots of two tiles");
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
IC_DEV int eff_groups(int groups, int64_t tiles) {
  const int64_t g = (tiles + kMinTiles - 1) / kMinTiles;
  return g < groups ? static_cast<int>(g) : groups;
}

template <bool FP8, bool SPARSE>
__global__ void __launch_bounds__(Cfg<FP8>::kThreads, 1)
    latent_attention_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kvmap,
                            const LatentArgs a) {
  using C = Cfg<FP8>;
  extern __shared__ __align__(1024) uint8_t smem[];
  // the swizzled layouts need a 1024-byte-aligned base
  if (smem_u32(smem) & 1023u) {
    if (threadIdx.x == 0) record_status(a.status, IC_ERR_UNSUPPORTED);
    return;
  }
  uint8_t* qs = smem + C::kOffQ;
  uint8_t* halves = smem + C::kOffHalf;
  uint8_t* ropes = smem + C::kOffRope;
  uint8_t* ps = smem + C::kOffP;
  uint8_t* raws = smem + C::kOffRaw;
  float* xm = reinterpret_cast<float*>(smem + C::kOffX);
  TileInfo* infos = reinterpret_cast<TileInfo*>(smem + C::kOffInfo);
  uint64_t* info_full = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  uint64_t* info_free = info_full + kInfo;
  uint64_t* half_full = info_free + kInfo;
  uint64_t* half_free = half_full + C::kHalves;
  uint64_t* rope_full = half_free + C::kHalves;
  uint64_t* rope_free = rope_full + C::kRopes;
  uint64_t* raw_full = rope_free + C::kRopes;
  uint64_t* raw_free = raw_full + C::kRaws;
  uint64_t* q_full = raw_free + C::kRaws;
  uint64_t* q_free = q_full + 1;   // the piece's last QK has read Q
  uint64_t* s_full = q_free + 1;   // [2] logits of a tile in TMEM
  uint64_t* p_ready = s_full + 2;  // weights of a tile in shared memory, O rescaled
  uint64_t* pv_done = p_ready + 1;
  uint64_t* o_free = pv_done + 1;  // a piece's output has been read out
  uint64_t* cleared = o_free + 1;  // bf16: the rows behind the end are zero
  uint64_t* xch = cleared + 1;     // softmax threads exchange a value
  uint64_t* retire = xch + 1;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 4);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int group = blockIdx.x / a.rblocks, rb = blockIdx.x - group * a.rblocks;
  pdl_trigger();
  if (threadIdx.x == 0) {
    tma_prefetch_desc(&qmap);
    if (!FP8) tma_prefetch_desc(&kvmap);
    for (int i = 0; i < kInfo; ++i) {
      mbar_init(&info_full[i], 1);
      mbar_init(&info_free[i], C::kReaders);
    }
    for (int i = 0; i < C::kHalves; ++i) {
      mbar_init(&half_full[i], FP8 ? 128 : 1);
      mbar_init(&half_free[i], 1);
    }
    for (int i = 0; i < C::kRopes; ++i) {
      mbar_init(&rope_full[i], FP8 ? 256 : 1);
      mbar_init(&rope_free[i], 1);
    }
    for (int i = 0; i < C::kRaws; ++i) {
      mbar_init(&raw_full[i], 1);
      mbar_init(&raw_free[i], 256);
    }
    mbar_init(q_full, 1);
    mbar_init(q_free, 1);
    mbar_init(&s_full[0], 1);
    mbar_init(&s_full[1], 1);
    mbar_init(p_ready, 128);
    mbar_init(pv_done, 1);
    mbar_init(o_free, 128);
    mbar_init(cleared, 32);
    mbar_init(xch, 128);
    mbar_init(retire, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  pdl_wait();
  if (warp == 1) {
    tmem_alloc(tmem_holder, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  const uint32_t kOutCol = 0, kSCol = 256;
  // one thread's wait, and a whole warp's: its lanes leave a wait that was
  // given up together, so that no lane stays behind in a warp-wide instruction
  auto wait1 = [&](uint64_t* bar, uint32_t parity) { return mbar_wait(bar, parity, abort_flag, a.status, a.wait_ns); };
  auto wait = [&](uint64_t* bar, uint32_t parity) { return __all_sync(0xffffffffu, wait1(bar, parity)) != 0; };
  // the descriptor of tile t, read by one thread or by a whole warp
  auto get_info1 = [&](int t, TileInfo& x) {
    if (!wait1(&info_full[t % kInfo], (t / kInfo) & 1)) return false;
    x = infos[t % kInfo];
    mbar_arrive(&info_free[t % kInfo]);
    return true;
  };
  auto get_info = [&](int t, TileInfo& x) {
    if (!wait(&info_full[t % kInfo], (t / kInfo) & 1)) return false;
    x = infos[t % kInfo];
    __syncwarp();
    if (lane == 0) mbar_arrive(&info_free[t % kInfo]);
    return true;
  };

  if (warp == 0) {
    // ------------------------------------------------------------ tiles and their copies
    // this group's share of all tiles
    int64_t total = 0;
    if (SPARSE) {
      total = static_cast<int64_t>(a.B) * tiles_of(a.k);
    } else {
      for (int b = lane; b < a.B; b += 32) {
        const int64_t n = a.lens[b];
        if (n != clamp_len(a, n)) record_status(a.status, IC_ERR_BAD_INDEX);
        total += tiles_of(static_cast<int>(clamp_len(a, n)));
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    }
    const int G = eff_groups(a.groups, total);
    const int64_t g0 = group < G ? group * total / G : 0;
    int64_t g1 = group < G ? (group + 1) * total / G : 0;
    // lane l holds the length of sequence cb + l
    int cb = 0, clen = 0;
    int64_t cstart = 0;  // first tile of sequence cb
    auto load_chunk = [&]() { clen = cb + lane < a.B ? seq_len<SPARSE>(a, cb + lane) : 0; };
    load_chunk();
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
    const int br = a.page_size % 64 == 0 ? 64 : a.page_size % 32 == 0 ? 32 : 16;  // rows of a TMA box
    const int run = br < kRawRows ? br : kRawRows;                                // rows of an e4m3 copy
    bool ok = true;
    int t = 0;
    int raw = 0, nrope = 0, nhalf = 0;  // e4m3 chunks, rotary slabs, latent halves issued
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
      // where the rows are: lane l finds the box (or copy, or row) l of the tile
      int64_t src = -1;   // e4m3: byte offset of the copy's first row
      int src_page = -1;  // bf16: page of the box
      int rows = 0;       // valid rows of the box
      int64_t src2 = -1;  // sparse: row 32 + lane
      const int unit = FP8 ? run : br;
      uint32_t m0 = 0, m1 = 0;
      if constexpr (SPARSE) {
        const int64_t num = static_cast<int64_t>(a.num_pages) * a.page_size;
        auto find = [&](int j) -> int64_t {
          if (j >= a.k) return -1;
          const int s = a.slots[static_cast<int64_t>(b) * a.k + j];
          if (s < 0 || s >= num) {
            if (s != -1) record_status(a.status, IC_ERR_BAD_INDEX);
            return -1;
          }
          const int page = s / a.page_size;
          return page * a.page_stride + static_cast<int64_t>(s - page * a.page_size) * kLatentRowFp8;
        };
        src = find(pos0 + lane);
        src2 = find(pos0 + 32 + lane);
        m0 = __ballot_sync(0xffffffffu, src >= 0);
        m1 = __ballot_sync(0xffffffffu, src2 >= 0);
      } else {
        const int p = pos0 + lane * unit;
        if (lane * unit < kT && p < blen) {
          const int pi = p / a.page_size;
          const int page = a.table[static_cast<int64_t>(b) * a.table_stride + pi];
          if (page >= 0 && page < a.num_pages) {
            rows = blen - p < unit ? blen - p : unit;
            src_page = page;
            src = page * a.page_stride + static_cast<int64_t>(p - pi * a.page_size) * kLatentRowFp8;
          } else {
            record_status(a.status, IC_ERR_BAD_INDEX);
          }
        }
        // bit r of the mask: row r is in a valid box, before the end
        const int rows_of = __shfl_sync(0xffffffffu, rows, lane / unit);
        const int rows_of2 = __shfl_sync(0xffffffffu, rows, (32 + lane) / unit);
        m0 = __ballot_sync(0xffffffffu, lane % unit < rows_of);
        m1 = __ballot_sync(0xffffffffu, (32 + lane) % unit < rows_of2);
      }
      if (!wait(&info_free[t % kInfo], ((t / kInfo) & 1) ^ 1)) {
        ok = false;
        break;
      }
      if (lane == 0) {
        TileInfo& x = infos[t % kInfo];
        x.b = b;
        x.pos0 = pos0;
        x.len = blen;
        x.mask[0] = m0;
        x.mask[1] = m1;
        // only a group's first piece starts at the group's start
        x.slot = 2 * group + (bstart <= g0 ? 0 : 1);
        x.flags = (first ? kFirst : 0) | (last ? kLast : 0) |
                  (bstart >= g0 && bstart + bt <= g1 ? kWhole : 0) | ((m0 & m1) != 0xffffffffu ? kClear : 0);
        mbar_arrive(&info_full[t % kInfo]);
      }
      if constexpr (FP8) {
        for (int c = 0; c < 2; ++c, ++raw) {
          const int rs = raw % C::kRaws;
          if (!wait(&raw_free[rs], ((raw / C::kRaws) & 1) ^ 1)) {
            ok = false;
            break;
          }
          uint8_t* dst = raws + rs * kRawBytes;
          const uint32_t bytes = static_cast<uint32_t>(__popc(c ? m1 : m0)) * kLatentRowFp8;
          if (lane == 0) {
            if (bytes) mbar_arrive_expect_tx(&raw_full[rs], bytes);
            else mbar_arrive(&raw_full[rs]);
          }
          __syncwarp();
          if constexpr (SPARSE) {
            const int64_t s = c ? src2 : src;
            if (s >= 0) bulk_load(dst + lane * kLatentRowFp8, a.cache + s, kLatentRowFp8, &raw_full[rs]);
          } else {
            const int l0 = c * (kRawRows / unit);  // lanes [l0, l0 + 32 / unit) have this chunk's copies
            if (lane >= l0 && lane < l0 + kRawRows / unit && rows > 0)
              bulk_load(dst + (lane - l0) * unit * kLatentRowFp8, a.cache + src,
                        static_cast<uint32_t>(rows) * kLatentRowFp8, &raw_full[rs]);
          }
        }
      } else {
        // boxes without a valid row read the page behind the last, which fills zeros
        const int pz = src_page >= 0 ? src_page : a.num_pages;
        const int py = (pos0 + lane * br) % a.page_size;
        const int rs = t % C::kRopes;
        if (!wait(&rope_free[rs], ((t / C::kRopes) & 1) ^ 1)) {
          ok = false;
          break;
        }
        if (lane == 0) mbar_arrive_expect_tx(&rope_full[rs], kSlab);
        __syncwarp();
        ++nrope;
        if (lane * br < kT) tma_load_3d(ropes + rs * kSlab + lane * br * 128, &kvmap, &rope_full[rs], 512, py, pz);
        for (int h = 0; h < 2; ++h) {
          const int hc = 2 * t + h, hs = hc % C::kHalves;
          if (!wait(&half_free[hs], ((hc / C::kHalves) & 1) ^ 1)) {
            ok = false;
            break;
          }
          if (lane == 0) mbar_arrive_expect_tx(&half_full[hs], kHalf);
          __syncwarp();
          ++nhalf;
          if (lane * br < kT)
#pragma unroll
            for (int c = 0; c < 4; ++c)
              tma_load_3d(halves + hs * kHalf + c * kSlab + lane * br * 128, &kvmap, &half_full[hs], h * 256 + c * 64,
                          py, pz);
        }
      }
    }
    if (ok) ok = wait(&info_free[n % kInfo], ((n / kInfo) & 1) ^ 1);
    if (ok && lane == 0) {
      infos[n % kInfo].flags = kEnd;
      mbar_arrive(&info_full[n % kInfo]);
    }
    // the last copies of each slot land before the CTA exits, whatever their readers do
    for (int u = raw > C::kRaws ? raw - C::kRaws : 0; u < raw; ++u)
      mbar_drain(&raw_full[u % C::kRaws], (u / C::kRaws) & 1);
    for (int u = nrope > C::kRopes ? nrope - C::kRopes : 0; u < nrope; ++u)
      mbar_drain(&rope_full[u % C::kRopes], (u / C::kRopes) & 1);
    for (int u = nhalf > C::kHalves ? nhalf - C::kHalves : 0; u < nhalf; ++u)
      mbar_drain(&half_full[u % C::kHalves], (u / C::kHalves) & 1);
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMAs
    if (elect_one()) {
      constexpr uint32_t idesc_qk = idesc_bf16_f32(64, 64, false, false);
      constexpr uint32_t idesc_pv = idesc_bf16_f32(64, 256, false, true);
      const uint32_t qa = smem_u32(qs), ha = smem_u32(halves), ra = smem_u32(ropes), pa = smem_u32(ps);
      int piece = -1, nclear = 0;  // piece of the tile whose PV comes next; cleared tiles seen
      // O += P . V of tile t
      auto pv = [&](int t, bool first) {
        if (first) {
          ++piece;
          if (piece > 0 && !wait1(o_free, (piece - 1) & 1)) return false;
        }
        if (!wait1(p_ready, t & 1)) return false;
        tc_fence_after();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t hs = (2 * t + h) % C::kHalves;
          const uint64_t vd = sw128_desc(ha + hs * kHalf, kSlab, 1024), pd = sw128_desc(pa, 16, 1024);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_ws_bf16_ss(tmem + kOutCol + h * 128, pd + kk * 2, vd + kk * 128, idesc_pv, !first || kk > 0);
          mma_commit(&half_free[hs]);
        }
        mma_commit(pv_done);
        return true;
      };
      int npieces = 0;
      bool prev_first = false;
      for (int t = 0;; ++t) {
        TileInfo x;
        if (!get_info1(t, x)) break;
        const bool end = (x.flags & kEnd) != 0, first = (x.flags & kFirst) != 0;
        // a piece's first QK waits for its Q, which is loaded once the last
        // piece's QK is done: that piece's last PV goes first
        if (C::kLag && t > 0 && (end || first) && !pv(t - 1, prev_first)) break;
        if (end) break;
        if (first) {
          if (!wait1(q_full, npieces & 1)) break;
          ++npieces;
        }
        if (!FP8 && (x.flags & kClear)) {
          if (!wait1(cleared, nclear & 1)) break;
          ++nclear;
        }
        const uint32_t d = tmem + kSCol + (t & 1) * 32;
        const int rs = t % C::kRopes;
        if (!wait1(&rope_full[rs], (t / C::kRopes) & 1)) break;
        tc_fence_after();
        {
          const uint64_t ad = sw128_desc(qa + 8 * kSlab, 16, 1024), bd = sw128_desc(ra + rs * kSlab, 16, 1024);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) mma_ws_bf16_ss(d, ad + kk * 2, bd + kk * 2, idesc_qk, kk > 0);
          mma_commit(&rope_free[rs]);
        }
        bool ok = true;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int hc = 2 * t + h, hs = hc % C::kHalves;
          if (ok && !wait1(&half_full[hs], (hc / C::kHalves) & 1)) ok = false;
          if (!ok) break;
          tc_fence_after();
          const uint64_t ad = sw128_desc(qa + h * 4 * kSlab, 16, 1024), bd = sw128_desc(ha + hs * kHalf, 16, 1024);
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_ws_bf16_ss(d, ad + c * (kSlab >> 4) + kk * 2, bd + c * (kSlab >> 4) + kk * 2, idesc_qk, 1);
        }
        if (!ok) break;
        mma_commit(&s_full[t & 1]);
        if (x.flags & kLast) mma_commit(q_free);
        if (C::kLag) {
          if (t > 0 && !first && !pv(t - 1, prev_first)) break;
          prev_first = first;
        } else if (!pv(t, first)) {
          break;
        }
      }
      // every MMA issued has retired before TMEM is released
      mma_commit(retire);
      mbar_drain(retire, 0);
    }
    __syncwarp();
  } else if (warp == 2) {
    // ------------------------------------------------------------ Q of each piece
    if (lane == 0) {
      int piece = 0;
      for (int t = 0;; ++t) {
        TileInfo x;
        if (!get_info1(t, x) || (x.flags & kEnd)) break;
        if (!(x.flags & kFirst)) continue;
        if (piece > 0 && !wait1(q_free, (piece - 1) & 1)) break;
        mbar_arrive_expect_tx(q_full, 9 * kSlab);
        const int row = x.b * a.rows + rb * 64;  // rows of the next sequence, or zeros, behind this one's: not written out
        for (int c = 0; c < 9; ++c) tma_load_2d(qs + c * kSlab, &qmap, q_full, c * 64, row);
        ++piece;
      }
      if (piece > 0) mbar_drain(q_full, (piece - 1) & 1);
    }
    __syncwarp();
  } else if (warp == 3) {
    // ------------------------------------------------------------ rows behind the end (bf16)
    if (!FP8) {
      for (int t = 0;; ++t) {
        TileInfo x;
        bool ok = get_info(t, x);
        if (!ok || (x.flags & kEnd)) break;
        if (!(x.flags & kClear)) continue;
        for (int h = 0; h < 2 && ok; ++h) {
          const int hc = 2 * t + h, hs = hc % C::kHalves;
          ok = wait(&half_full[hs], (hc / C::kHalves) & 1);
          if (!ok) break;
          const uint32_t base = smem_u32(halves + hs * kHalf) + (lane >> 3) * kSlab + (lane & 7) * 16;
          for (int r = 0; r < kT; ++r)
            if (!((x.mask[r >> 5] >> (r & 31)) & 1u)) st_shared_v4(base + r * 128, make_uint4(0, 0, 0, 0));
        }
        if (!ok) break;
        fence_proxy_async_smem();
        mbar_arrive(cleared);
      }
    }
  } else if (warp < 8) {
    // ------------------------------------------------------------ softmax and output
    // Thread (quadrant, lane) has query row r of the block and one half of the
    // columns: 32 of a tile's keys, 256 of the output dims.
    const int quad = warp & 3, colh = quad >> 1;
    const int r = (quad & 1) * 32 + lane;
    const int tid = quad * 32 + lane;
    const uint32_t tlane = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    const float c2 = a.sm_scale * kLog2e;
    const int row = rb * 64 + r;             // query row of the sequence
    const bool live = row < a.rows;
    const int back = a.Q - 1 - (live ? row / a.H : 0);  // the row's token ends this many positions before the last
    const float sink2 = a.sink && live ? a.sink[row % a.H] * kLog2e : -INFINITY;
    float ref = -INFINITY, l = 0.f;
    uint32_t nx = 0;  // exchanges so far
    auto exchange = [&](float v, float& other) {
      float* buf = xm + (nx & 1) * 128;
      buf[tid] = v;
      mbar_arrive(xch);
      const bool ok = wait(xch, nx & 1);
      ++nx;
      other = buf[tid ^ 64];
      return ok;
    };
    for (int t = 0;; ++t) {
      TileInfo x;
      bool ok = get_info(t, x);
      if (!ok || (x.flags & kEnd)) break;
      ok = wait(&s_full[t & 1], (t >> 1) & 1);
      if (!ok) break;
      tc_fence_after();
      uint32_t rv[32];
      tmem_ld32_issue(tlane + kSCol + (t & 1) * 32, rv);
      if (x.flags & kFirst) {
        ref = -INFINITY;
        l = 0.f;
      }
      uint32_t mask = x.mask[colh];
      const int seen = x.len - back - (x.pos0 + colh * 32);  // columns of this thread before the row's limit
      if (seen < 32) mask = seen <= 0 ? 0u : mask & ((1u << seen) - 1);
      tmem_ld_wait(rv);
      if (!__all_sync(0xffffffffu, mask == 0xffffffffu)) {
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (!((mask >> j) & 1u)) rv[j] = 0xff800000u;  // -inf
      }
      float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int j = 0; j < 32; ++j) mx[j & 3] = fmaxf(mx[j & 3], __uint_as_float(rv[j]));
      const float mine = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
      float other;
      ok = exchange(mine, other);
      if (!ok) break;
      const float m = fmaxf(mine, other) * c2;
      // the reference moves when the row's maximum passes it by more than
      // kMove: weights stay below 2^8, far from bf16's and fp32's limits
      float scale = 1.f;
      if (ref == -INFINITY) {
        ref = m;
      } else if (m > ref + kMove) {
        scale = ex2_approx(ref - m);
        ref = m;
      }
      const float base = ref == -INFINITY ? 0.f : ref;  // nothing valid so far: every weight is 0
      uint32_t pk[16];
      float sum[4] = {0.f, 0.f, 0.f, 0.f};
      // the sum is of the 32-bit weights; those of the product are rounded to
      // bf16 (2^-8 of each at most, of either sign), as the MMA takes them
#pragma unroll
      for (int j = 0; j < 32; j += 2) {
        const float p0 = ex2_approx(fmaf(__uint_as_float(rv[j]), c2, -base));
        const float p1 = ex2_approx(fmaf(__uint_as_float(rv[j + 1]), c2, -base));
        sum[(j >> 1) & 3] += p0 + p1;
        pk[j >> 1] = pack_bf16x2(p0, p1);
      }
      l = fmaf(l, scale, (sum[0] + sum[1]) + (sum[2] + sum[3]));
      // the previous PV has read the weights, and O stands still
      if (t > 0) ok = wait(pv_done, (t - 1) & 1);
      if (!ok) break;
      if (__any_sync(0xffffffffu, scale != 1.f)) {
        tc_fence_after();
#pragma unroll 1
        for (int c = 0; c < 8; ++c) {
          uint32_t o[32];
          tmem_ld32_issue(tlane + kOutCol + c * 32, o);
          tmem_ld_wait(o);
#pragma unroll
          for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * scale);
          tmem_st32(tlane + kOutCol + c * 32, o);
        }
        tmem_st_wait();
      }
      const uint32_t pb = smem_u32(ps);
#pragma unroll
      for (int q4 = 0; q4 < 4; ++q4)
        st_shared_v4(pb + sw128_offset(r, colh * 4 + q4),
                     make_uint4(pk[4 * q4], pk[4 * q4 + 1], pk[4 * q4 + 2], pk[4 * q4 + 3]));
      fence_proxy_async_smem();
      tc_fence_before();
      mbar_arrive(p_ready);
      if (!(x.flags & kLast)) continue;
      // ---- the piece's output
      float l2;
      ok = exchange(l, l2) && wait(pv_done, t & 1);
      if (!ok) break;
      tc_fence_after();
      const float lsum = l + l2;
      const bool whole = (x.flags & kWhole) != 0;
      const int64_t gr = (static_cast<int64_t>(x.b) * a.rows) + row;
      const int64_t pr = (static_cast<int64_t>(x.slot) * a.rblocks + rb) * 64 + r;
      float f = 1.f;
      if (whole) {
        const float M = fmaxf(ref, sink2);
        const float w = ref == -INFINITY ? 0.f : exp2f(ref - M);
        const float den = lsum * w + (sink2 == -INFINITY ? 0.f : exp2f(sink2 - M));
        f = w > 0.f ? w / den : 0.f;
        if (live && colh == 0 && a.lse) a.lse[gr] = M == -INFINITY ? -INFINITY : (M + log2f(den)) / kLog2e;
      } else if (colh == 0) {
        a.part_ml[pr * 2] = ref;
        a.part_ml[pr * 2 + 1] = lsum;
      }
#pragma unroll 1
      for (int c = 0; c < 8; ++c) {
        uint32_t o[32];
        tmem_ld32_issue(tlane + kOutCol + c * 32, o);
        tmem_ld_wait(o);
        const int dim = (c >> 2) * 256 + colh * 128 + (c & 3) * 32;
        if (!whole) {
          uint4* dst = reinterpret_cast<uint4*>(a.part_o + pr * 512 + dim);
#pragma unroll
          for (int k = 0; k < 8; ++k) dst[k] = make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
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
      mbar_arrive(o_free);
    }
  } else if (FP8) {
    // ------------------------------------------------------------ widening (e4m3)
    // Warp w has the 64 dims of slab w: eight rows x four 16-code words a step
    // (a staged row is 41 words long, an odd number: eight rows of one word
    // column lie in eight different bank groups), and one rotary word a thread.
    const int w = warp - 8, ct = threadIdx.x - 256;
    int raw = 0;
    for (int t = 0;; ++t) {
      TileInfo x;
      bool ok = get_info(t, x);
      if (!ok || (x.flags & kEnd)) break;
      const int rs = t % C::kRopes, hc = 2 * t + (w >> 2), hs = hc % C::kHalves;
      ok = wait(&rope_free[rs], ((t / C::kRopes) & 1) ^ 1) &&
           wait(&half_free[hs], ((hc / C::kHalves) & 1) ^ 1);
      const uint32_t slab = smem_u32(halves + hs * kHalf + (w & 3) * kSlab);
      const uint32_t rope = smem_u32(ropes + rs * kSlab);
      for (int c = 0; c < 2 && ok; ++c, ++raw) {
        const int ws = raw % C::kRaws;
        ok = wait(&raw_full[ws], (raw / C::kRaws) & 1);
        if (!ok) break;
        const uint8_t* src = raws + ws * kRawBytes;
        const uint32_t mask = x.mask[c];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int rr = (lane & 7) + 8 * j, ch = lane >> 3;
          const uint8_t* rowp = src + rr * kLatentRowFp8;
          uint32_t o[8] = {0, 0, 0, 0, 0, 0, 0, 0};
          if ((mask >> rr) & 1u)
            e4m3x16_to_bf16x16(*reinterpret_cast<const uint4*>(rowp + w * 64 + ch * 16),
                               *reinterpret_cast<const float*>(rowp + 512 + (w >> 1) * 4), o);
          const int row = c * 32 + rr;
          st_shared_v4(slab + sw128_offset(row, 2 * ch), make_uint4(o[0], o[1], o[2], o[3]));
          st_shared_v4(slab + sw128_offset(row, 2 * ch + 1), make_uint4(o[4], o[5], o[6], o[7]));
        }
        {
          const int rr = ct >> 3, ch = ct & 7;
          uint4 v = make_uint4(0, 0, 0, 0);
          if ((mask >> rr) & 1u) v = *reinterpret_cast<const uint4*>(src + rr * kLatentRowFp8 + 528 + ch * 16);
          st_shared_v4(rope + sw128_offset(c * 32 + rr, ch), v);
        }
        mbar_arrive(&raw_free[ws]);
      }
      if (!ok) break;
      fence_proxy_async_smem();
      mbar_arrive(&rope_full[rs]);
      mbar_arrive(&half_full[hs]);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the pieces of each sequence that more than one group worked on, and
// writes the rows of sequences without a tile. WPR warps share a row's pieces;
// lane l has dims 128 i + 4 l + [0, 4), i < 4.
constexpr int kJoinThreads = 256;
template <bool SPARSE, int WPR>
__global__ void __launch_bounds__(kJoinThreads) latent_join_kernel(const LatentArgs a) {
  constexpr int RPC = 8 / WPR;  // rows of a CTA
  __shared__ int64_t sums[2][8];
  __shared__ float4 accs[WPR > 1 ? 8 : 1][128];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per_seq = (a.rows + RPC - 1) / RPC;
  const int b = blockIdx.x / per_seq;
  const int row = (blockIdx.x - b * per_seq) * RPC + warp / WPR;
  pdl_trigger();
  pdl_wait();
  // tiles of all sequences, and of those before b
  int64_t total = 0, start = 0;
  int bt;
  if (SPARSE) {
    bt = tiles_of(a.k);
    total = static_cast<int64_t>(a.B) * bt;
    start = static_cast<int64_t>(b) * bt;
  } else {
    for (int i = threadIdx.x; i < a.B; i += kJoinThreads) {
      const int n = tiles_of(seq_len<SPARSE>(a, i));
      total += n;
      if (i < b) start += n;
    }
    bt = tiles_of(seq_len<SPARSE>(a, b));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      total += __shfl_xor_sync(0xffffffffu, total, o);
      start += __shfl_xor_sync(0xffffffffu, start, o);
    }
    if (lane == 0) {
      sums[0][warp] = total;
      sums[1][warp] = start;
    }
    __syncthreads();
    total = start = 0;
    for (int i = 0; i < 8; ++i) {
      total += sums[0][i];
      start += sums[1][i];
    }
  }
  int gf = 0, gl = -1;
  const int G = eff_groups(a.groups, total);
  if (bt > 0) {
    gf = static_cast<int>(((start + 1) * G - 1) / total);  // the group of the first tile, and of the last
    gl = static_cast<int>(((start + bt) * G - 1) / total);
    if (gf == gl) return;  // one piece: written already
  }
  const bool live = row < a.rows;
  const int rb = row >> 6, r = row & 63;
  auto part_row = [&](int g) {
    const int slot = 2 * g + (g * total / G >= start ? 0 : 1);
    return (static_cast<int64_t>(slot) * a.rblocks + rb) * 64 + r;
  };
  const float sink2 = a.sink && live ? a.sink[row % a.H] * kLog2e : -INFINITY;
  float M = sink2, den = 0.f;
  float4 acc[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  if (live) {
    const float2* ml = reinterpret_cast<const float2*>(a.part_ml);
    for (int g = gf + lane; g <= gl; g += 32) M = fmaxf(M, ml[part_row(g)].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    for (int g = gf + lane; g <= gl; g += 32) {
      const float2 v = ml[part_row(g)];
      if (v.x != -INFINITY) den = fmaf(exp2f(v.x - M), v.y, den);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) den += __shfl_xor_sync(0xffffffffu, den, o);
    if (sink2 != -INFINITY) den += exp2f(sink2 - M);
#pragma unroll 4
    for (int g = gf + warp % WPR; g <= gl; g += WPR) {
      const int64_t pr = part_row(g);
      const float m = ml[pr].x;
      const float w = m == -INFINITY ? 0.f : exp2f(m - M);
      const float4* src = reinterpret_cast<const float4*>(a.part_o + pr * 512) + lane;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 v = src[32 * i];
        acc[i].x = fmaf(w, v.x, acc[i].x);
        acc[i].y = fmaf(w, v.y, acc[i].y);
        acc[i].z = fmaf(w, v.z, acc[i].z);
        acc[i].w = fmaf(w, v.w, acc[i].w);
      }
    }
  }
  if constexpr (WPR > 1) {
#pragma unroll
    for (int i = 0; i < 4; ++i) accs[warp][32 * i + lane] = acc[i];
    __syncthreads();
    if (warp % WPR) return;
    for (int k = 1; k < WPR; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 v = accs[warp + k][32 * i + lane];
        acc[i].x += v.x;
        acc[i].y += v.y;
        acc[i].z += v.z;
        acc[i].w += v.w;
      }
  }
  if (!live) return;
  const float inv = den > 0.f ? 1.f / den : 0.f;
  const int64_t gr = static_cast<int64_t>(b) * a.rows + row;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float o[4] = {acc[i].x * inv, acc[i].y * inv, acc[i].z * inv, acc[i].w * inv};
    const int dim = 128 * i + 4 * lane;
    if (a.gate) {
      const uint2 g = *reinterpret_cast<const uint2*>(a.gate + gr * 512 + dim);
      const uint32_t gw[2] = {g.x, g.y};
#pragma unroll
      for (int e = 0; e < 4; ++e)
        o[e] *= __fdividef(1.f, 1.f + ex2_approx(-kLog2e * bf16_lane(gw[e >> 1], e & 1)));
    }
    if (a.out_f32)
      *reinterpret_cast<float4*>(static_cast<float*>(a.out) + gr * 512 + dim) = make_float4(o[0], o[1], o[2], o[3]);
    else
      *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + gr * 512 + dim) =
          make_uint2(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]));
  }
  if (a.lse && lane == 0) a.lse[gr] = M == -INFINITY ? -INFINITY : (M + log2f(den)) / kLog2e;
}

template <bool FP8, bool SPARSE>
cudaError_t launch_main(const CUtensorMap& qmap, const CUtensorMap& kvmap, const LatentArgs& a, cudaStream_t stream) {
  using C = Cfg<FP8>;
  auto kern = latent_attention_kernel<FP8, SPARSE>;
  static bool done[64] = {false};
  cudaError_t e = set_smem_once(kern, C::kSmemBytes, done);
  if (e != cudaSuccess) return e;
  return launch_kernel(kern, dim3(static_cast<unsigned>(a.groups) * a.rblocks), dim3(C::kThreads), C::kSmemBytes,
                       stream, false, qmap, kvmap, a);
}

template <bool SPARSE>
cudaError_t launch_join(const LatentArgs& a, cudaStream_t stream) {
  // pieces of a sequence: about groups / B + 1
  const int pieces = a.groups / a.B + 1;
  const int wpr = pieces <= 2 ? 1 : pieces <= 8 ? 4 : 8;
  const int rpc = 8 / wpr;
  const dim3 grid(static_cast<unsigned>(a.B) * ((a.rows + rpc - 1) / rpc));
  auto kern = wpr == 1 ? latent_join_kernel<SPARSE, 1>
                       : wpr == 4 ? latent_join_kernel<SPARSE, 4> : latent_join_kernel<SPARSE, 8>;
  return launch_kernel(kern, grid, dim3(kJoinThreads), 0, stream, true, a);
}

}  // namespace

cudaError_t launch_latent_attention(const CUtensorMap& qmap, const CUtensorMap& kvmap, const LatentArgs& a, bool fp8,
                                    bool sparse, cudaStream_t stream, int* launches) {
  cudaError_t e = sparse ? launch_main<true, true>(qmap, kvmap, a, stream)
                  : fp8  ? launch_main<true, false>(qmap, kvmap, a, stream)
                         : launch_main<false, false>(qmap, kvmap, a, stream);
  if (e != cudaSuccess) return e;
  e = sparse ? launch_join<true>(a, stream) : launch_join<false>(a, stream);
  if (e != cudaSuccess) return e;
  *launches += 2;
  return cudaGetLastError();
}

}  // namespace ic
