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
// each block of query rows (32 rows, or 64 of 33 to 64; above that pairs of CTAs
// take 128, latent_pair.cu). A piece is what one group has of one sequence:
// whole sequences are finished by their CTA, the others leave (reference, sum,
// unnormalised output) in fp32 and a second kernel joins them.
//
// CTA. M query rows in the weight-stationary MMA form. M = 32: lane quadrant q
// of TMEM holds the 32 rows' columns [q N / 4, (q + 1) N / 4), and Q, an operand
// in TMEM, is there once in each quadrant; it enters through a tile's stage, so
// that three tiles fit. M = 64: lanes 0-63 hold the first half of the columns,
// 64-127 the second; Q stays in shared memory (72 KB) beside two tiles. Per tile
//   S[M x 64]   = Q . K^T         (36 MMAs, N = 64)
//   P           = 2^(S sm_scale log2e - ref), bf16 into shared memory
//   O[M x 512] += P . V           (8 MMAs, N = 256; V is the same tile read
//                                  as an MN-major operand)
// with the running reference of an online softmax, moved (and O rescaled) only
// when a row's maximum passes it by more than 2^8.
//
// What bounds it. The MMAs of a tile take 1600 cycles at M = 32 (28 and 76 a
// product, measured) and 1800 at M = 64 (32 and 80); the bytes of an e4m3 tile,
// 42 KB, are 1800 cycles of an SM's share of HBM. Measured, a tile takes 3000
// cycles of e4m3 (4 sequences of 54K rows on average, 32 query rows: 65 us with
// 8 us of joining; 2.5 TB/s before it): the widening warps need 1200 of issue alone, and the
// rest is the latency of their chain (descriptor, loads, conversion, stores, fence)
// with two warps a scheduler. Converting with a quarter fewer instructions, and
// counting the rings' places along instead of dividing, gave 3 % together; a second
// set of widening warps has no registers left. A bf16 tile takes as long as its
// chain QK -> softmax -> PV, of which two tiles are under way. Small calls (one
// sequence of a few hundred rows, 12 us) are two launches, the setup of a CTA
// (barriers, TMEM, lengths: 5000 cycles to the first product), one tile and the join.
//
// Roles. Warp 0 finds the tiles, up to kInfo ahead, and asks L2 for them;
// warps 1 and 2 issue the two products, each as soon as its own inputs are
// there; warps 4-7 load Q and run the softmax and the output. bf16 pages: warp
// 3 issues TMA boxes that land in the operand layout, warp 8 clears the rows
// behind a sequence's end (a zero weight times a NaN left there would be NaN).
// e4m3 pages: warps 8-15 take a tile's codes to registers, straight from L2, and
// widen them into the operand layout (there is no room to stage them in shared
// memory).
#include "latent.cuh"

namespace ic {

namespace {

template <bool FP8, bool SPARSE, int M>
struct Cfg {
  using R = Rows<M>;
  static constexpr int kThreads = FP8 ? 512 : 288;
  // tile descriptors in flight; a sparse one has its 64 rows' places with it
  static constexpr int kInfo = SPARSE ? 3 : 8;
  static constexpr int kOffQ = R::kStages * kTile;  // M = 64
  static constexpr int kOffP = kOffQ + (R::kQStage ? 0 : 9 * R::kQSlab);
  static constexpr int kOffX = kOffP + R::kPBufs * R::kP;  // [2][128] row maxima / sums
  static constexpr int kOffInfo = kOffX + 2 * 128 * 4;
  static constexpr int kOffSlots = kOffInfo + kInfo * static_cast<int>(sizeof(TileInfo));
  static constexpr int kOffBar = kOffSlots + (SPARSE ? kInfo * kT * 8 : 0);
  // readers of a tile descriptor: the two issuing warps, four softmax warps, and
  // the copying and the clearing warp or the widening warps
  static constexpr int kReaders = 6 + (FP8 ? 8 : 2);
  static constexpr int kNumBars = 2 * kInfo + 2 * R::kStages + 12 + R::kClears;
  static constexpr int kOffMisc = kOffBar + kNumBars * 8;
  static constexpr int kSmemBytes = kOffMisc + 16;
  static_assert(kOffBar % 8 == 0, "alignment");
  static_assert(kSmemBytes <= 232448, "fits one CTA per SM");
};

template <bool FP8, bool SPARSE, int M>
__global__ void __launch_bounds__(Cfg<FP8, SPARSE, M>::kThreads, 1)
    latent_attention_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kvmap,
                            const LatentArgs a) {
  using C = Cfg<FP8, SPARSE, M>;
  using R = Rows<M>;
  constexpr int kInfo = C::kInfo, kStages = R::kStages, kClears = R::kClears, kCols = R::kCols, kDims = R::kDims;
  constexpr uint32_t kOutCol = R::kOutCol, kSCol = R::kSCol, kQCol = R::kQCol;
  constexpr bool kQStage = R::kQStage;
  extern __shared__ __align__(1024) uint8_t smem[];
  // the swizzled layouts need a 1024-byte-aligned base
  if (smem_u32(smem) & 1023u) {
    if (threadIdx.x == 0) record_status(a.status, IC_ERR_UNSUPPORTED);
    return;
  }
  uint8_t* qs = smem + C::kOffQ;
  uint8_t* ps = smem + C::kOffP;
  float* xm = reinterpret_cast<float*>(smem + C::kOffX);
  TileInfo* infos = reinterpret_cast<TileInfo*>(smem + C::kOffInfo);
  int64_t* places = reinterpret_cast<int64_t*>(smem + C::kOffSlots);  // sparse: [kInfo][64] byte offsets in the cache
  uint64_t* info_full = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  uint64_t* info_free = info_full + kInfo;
  // the stages hold, in order, each piece's Q (M = 32) and its tiles
  uint64_t* full = info_free + kInfo;  // [kStages] Q as loaded, or a tile in operand layout
  uint64_t* freed = full + kStages;    // [kStages] Q is in TMEM, or the tile's last product has read it (bf16: and warp 8 has seen it)
  uint64_t* q_full = freed + kStages;
  uint64_t* q_free = q_full + 1;    // the piece's last QK has read Q
  uint64_t* s_full = q_free + 1;    // [2] logits of a tile in TMEM
  uint64_t* p_ready = s_full + 2;   // [2] weights of a tile in shared memory, its logits read, O rescaled
  uint64_t* pv_done = p_ready + 2;  // [2]
  uint64_t* o_free = pv_done + 2;   // a piece's output has been read out
  uint64_t* cleared = o_free + 1;   // [kClears] bf16: a tile's rows that hold nothing are zero
  uint64_t* xch = cleared + kClears;  // [2] the softmax warps that share rows exchange a value
  uint64_t* retire = xch + 2;
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
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&full[i], FP8 ? 8 : 1);
      mbar_init(&freed[i], FP8 ? 1 : 2);
    }
    mbar_init(q_full, kQStage ? 4 : 1);
    mbar_init(q_free, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_ready[i], 4);
      mbar_init(&pv_done[i], 1);
    }
    mbar_init(o_free, 4);
    for (int i = 0; i < kClears; ++i) mbar_init(&cleared[i], 1);
    mbar_init(&xch[0], R::kParts);
    mbar_init(&xch[1], R::kParts);
    mbar_init(retire, 2);
    *abort_flag = 0;
    fence_mbar_init();
  }
  pdl_wait();
  const int64_t len0 = !SPARSE && warp == 0 && lane < a.B ? a.lens[lane] : 0;
  if (warp == 1) {
    tmem_alloc(tmem_holder, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  // A whole warp waits: its lanes leave a wait that was given up together, so
  // that no lane stays behind in a warp-wide instruction. (A lane that waits
  // alone wakes late: 430 to 690 cycles after the arrival against 120 to 140,
  // measured with 2 to 24 waiting warps.)
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait_hot(bar, parity, abort_flag, a.status, a.wait_ns)) != 0;
  };
  // one arrival for the warp, after all its lanes' writes. (The lanes meet
  // again before any of them can enter a wait: a try suspends the warp, and the
  // one lane's work would wait with it.)
  auto warp_arrive = [&](uint64_t* bar) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
    __syncwarp();
  };
  // the descriptor of tile t
  auto get_info = [&](int t, TileInfo& x) {
    if (!wait(&info_full[t % kInfo], (t / kInfo) & 1)) return false;
    x = infos[t % kInfo];
    warp_arrive(&info_free[t % kInfo]);
    return true;
  };
  // Q's rows of sequence b, by one warp. (Rows of the next sequence, or zeros,
  // may lie behind this one's: they are not written out.) One elected lane
  // issues the copies: lanes that issue their own cost about 100 cycles each.
  auto copy_q = [&](int b, uint8_t* dst, uint64_t* bar) {
    if (elect_one()) {
#pragma unroll
      for (int c = 0; c < 9; ++c) tma_load_2d(dst + c * R::kQSlab, &qmap, bar, c * 64, b * a.rows + rb * M);
    }
    __syncwarp();
  };
  const int br = a.page_size % 64 == 0 ? 64 : a.page_size % 32 == 0 ? 32 : 16;  // rows of a TMA box

  // (One branch for each four warps: in a chain of single warps' the compiler spills
  // in the softmax, whose reloads past the L1 that 227 KB leave cost a quarter of the
  // e4m3 batch's time.)
  if (warp < 4) {
    if (warp == 0) {
      // ------------------------------------------------------------ tiles
      find_tiles<FP8, SPARSE, kInfo>(a, len0, group, FP8 ? 16 : br, -1, infos, places, info_full, info_free, wait);
    } else if (warp == 1) {
      // ------------------------------------------------------------ S = Q . K^T
      constexpr uint32_t idesc = idesc_bf16_f32(M, kT, false, false);
      const uint32_t ka = smem_u32(smem);
      int pieces = 0, n = 0;  // stages used so far
#pragma unroll 1
      for (int t = 0;; ++t, ++n) {
        TileInfo x;
        if (!get_info(t, x) || (x.flags & kEnd)) break;
        if (x.flags & kFirst) {
          if (!kQStage) {
            if (pieces > 0 && !wait(q_free, (pieces - 1) & 1)) break;
            if (lane == 0) mbar_arrive_expect_tx(q_full, 9 * R::kQSlab);
            __syncwarp();
            copy_q(x.b, qs, q_full);
          }
          ++pieces;
          if (!wait(q_full, (pieces - 1) & 1)) break;
          if (kQStage) {
            if (lane == 0) mbar_arrive(&freed[n % kStages]);
            __syncwarp();
            ++n;
          }
        }
        // the logits of tile t - 2 have been read
        if (t >= 2 && !wait(&p_ready[t & 1], ((t >> 1) - 1) & 1)) break;
        const int st = n % kStages;
        if (!wait(&full[st], (n / kStages) & 1)) break;
        tc_fence_after();
        if (elect_one()) {
          const uint32_t d = tmem + kSCol + (t & 1) * kCols;
          const uint64_t bd = sw128_desc(ka + st * kTile, 16, 1024), ad = sw128_desc(smem_u32(qs), 16, 1024);
#pragma unroll 1
          for (int c = 0; c < 9; ++c)
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
              if constexpr (kQStage)
                mma_ws_bf16_ts(d, tmem + kQCol + c * 32 + kk * 8, bd + c * (kSlab >> 4) + kk * 2, idesc, c + kk > 0);
              else
                mma_ws_bf16_ss(d, ad + c * (R::kQSlab >> 4) + kk * 2, bd + c * (kSlab >> 4) + kk * 2, idesc, c + kk > 0);
            }
          mma_commit(&s_full[t & 1]);
          if (x.flags & kLast) mma_commit(q_free);
        }
        __syncwarp();
      }
      // every MMA issued has retired before TMEM is released (the lane that
      // elect_one names is the same each time)
      if (elect_one()) mma_commit(retire);
      __syncwarp();
      mbar_drain(retire, 0);
      if (!kQStage && pieces > 0) mbar_drain(q_full, (pieces - 1) & 1);  // given up: Q lands before the CTA exits
    } else if (warp == 2) {
      // ------------------------------------------------------------ O += P . V
      constexpr uint32_t idesc = idesc_bf16_f32(M, 256, false, true);
      const uint32_t va = smem_u32(smem), pa = smem_u32(ps);
      int pieces = 0, nclear = 0, n = 0;
#pragma unroll 1
      for (int t = 0;; ++t, ++n) {
        TileInfo x;
        if (!get_info(t, x) || (x.flags & kEnd)) break;
        const bool first = (x.flags & kFirst) != 0;
        if (first) {
          if (pieces > 0 && !wait(o_free, (pieces - 1) & 1)) break;
          ++pieces;
          if (kQStage) ++n;
        }
        if (!FP8 && (x.flags & kClear)) {
          if (!wait(&cleared[nclear % kClears], (nclear / kClears) & 1)) break;
          ++nclear;
        }
        const int st = n % kStages;
        if (!wait(&full[st], (n / kStages) & 1)) break;
        if (!wait(&p_ready[t & 1], (t >> 1) & 1)) break;
        tc_fence_after();
        if (elect_one()) {
          const uint64_t vd = sw128_desc(va + st * kTile, kSlab, 1024), pd = sw128_desc(pa + (t % R::kPBufs) * R::kP, 16, 1024);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
#pragma unroll
            for (int h = 0; h < 2; ++h)
              mma_ws_bf16_ss(tmem + kOutCol + h * kDims, pd + kk * 2, vd + h * (4 * kSlab >> 4) + kk * 128, idesc,
                             !first || kk > 0);
          mma_commit(&freed[st]);
          mma_commit(&pv_done[t & 1]);
        }
        __syncwarp();
      }
      if (elect_one()) mma_commit(retire);
      __syncwarp();
      mbar_drain(retire, 0);
    } else if (warp == 3) {
      // ------------------------------------------------------------ copies (bf16)
      // The stages have one producer that fills them in order: a second one that
      // ran ahead would take the parity of an older phase for its own.
      if (!FP8) {
        int n = 0;
        auto stage = [&](uint32_t bytes) {  // the next stage, ready for copies of so many bytes
          if (!wait(&freed[n % kStages], ((n / kStages) & 1) ^ 1)) return false;
          if (lane == 0) mbar_arrive_expect_tx(&full[n % kStages], bytes);
          __syncwarp();
          return true;
        };
        for (int t = 0;; ++t) {
          TileInfo x;
          if (!get_info(t, x) || (x.flags & kEnd)) break;
          if (kQStage && (x.flags & kFirst)) {
            if (!stage(9 * R::kQSlab)) break;
            copy_q(x.b, smem + (n % kStages) * kTile, &full[n % kStages]);
            ++n;
          }
          if (!stage(kTile)) break;
          // boxes without a valid row read the page behind the last, which fills zeros
          if (elect_one()) {
            uint8_t* dst = smem + (n % kStages) * kTile;
            int py = x.row0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              if (i * br >= kT) break;
              const int pz = x.at[i] < 0 ? a.num_pages : static_cast<int>(x.at[i]);
#pragma unroll
              for (int c = 0; c < 9; ++c)
                tma_load_3d(dst + c * kSlab + i * br * 128, &kvmap, &full[n % kStages], c * 64, py, pz);
              py += br;
              if (py >= a.page_size) py = 0;
            }
          }
          __syncwarp();
          ++n;
        }
        // the last copies of each stage land before the CTA exits, whatever their readers do
        for (int u = n > kStages ? n - kStages : 0; u < n; ++u)
          if (lane == 0) mbar_drain(&full[u % kStages], (u / kStages) & 1);
        __syncwarp();
      }
    }
  } else if (warp < 8) {
    // ------------------------------------------------------------ Q, softmax and output
    // Q of a piece from its stage into the quadrant's copy in TMEM
    int n = 0;
    auto load_q = [&](uint32_t tlane) {
      if (!kQStage) return true;
      if (!wait(&full[n % kStages], (n / kStages) & 1)) return false;
      const uint8_t* src = smem + (n % kStages) * kTile;
#pragma unroll 1
      for (int c = 0; c < 9; ++c) {
        uint32_t v[32];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint4 w = *reinterpret_cast<const uint4*>(src + c * R::kQSlab + sw128_offset(lane, i));
          v[4 * i] = w.x;
          v[4 * i + 1] = w.y;
          v[4 * i + 2] = w.z;
          v[4 * i + 3] = w.w;
        }
        tmem_st32(tlane + kQCol + c * 32, v);
      }
      tmem_st_wait();
      tc_fence_before();
      warp_arrive(q_full);
      ++n;
      return true;
    };
    softmax_rows<M, false>(a, tmem, ps, xm, s_full, pv_done, q_free, xch, rb * M, rb, wait, warp_arrive,
                           [&](int t, TileInfo& x) {
                             if (t > 0) ++n;  // tile t - 1 has taken a stage
                             return get_info(t, x);
                           },
                           load_q, [&](int t) { warp_arrive(&p_ready[t & 1]); }, [&]() { warp_arrive(o_free); });
  } else if (!FP8) {
    // ------------------------------------------------------------ rows behind the end (bf16)
    // Every stage passes through this warp, with something to clear or not, and
    // is freed by it too: a wait for a stage some phases ahead, or behind, would
    // take another phase of the same parity for its own.
    int n = 0, nclear = 0;
    auto landed = [&]() { return wait(&full[n % kStages], (n / kStages) & 1); };
    for (int t = 0;; ++t, ++n) {
      TileInfo x;
      if (!get_info(t, x) || (x.flags & kEnd)) break;
      if (kQStage && (x.flags & kFirst)) {
        if (!landed()) break;
        warp_arrive(&freed[n % kStages]);
        ++n;
      }
      if (!landed()) break;
      const int st = n % kStages;
      if (x.flags & kClear) {
        const uint32_t base = smem_u32(smem) + st * kTile + (lane >> 3) * kSlab + (lane & 7) * 16;
#pragma unroll 8
        for (int r = 0; r < kT; ++r)
          if (!(((r & 32 ? x.mask[1] : x.mask[0]) >> (r & 31)) & 1u)) {
            st_shared_v4(base + r * 128, make_uint4(0, 0, 0, 0));
            st_shared_v4(base + 4 * kSlab + r * 128, make_uint4(0, 0, 0, 0));
          }
        fence_proxy_async_smem();
        warp_arrive(&cleared[nclear % kClears]);
        ++nclear;
      }
      warp_arrive(&freed[st]);
    }
  } else {
    // ------------------------------------------------------------ widening (e4m3)
    // Warp w has eight rows of the tile, in two units of four. A load takes a
    // whole row's codes, lane l the 16 of word l: four lines an instruction
    // (64-byte pieces of eight rows cost four times the lookups in L1, which then
    // bound the kernel). Eight lanes that store together have four words of two
    // neighbouring slabs; those of the odd slab store their second half first, so
    // the eight meet eight chunks of the swizzle. Both units are on their way at
    // once: one's next loads are issued as soon as its registers are read.
    const int w = warp - 8;
    struct Unit {
      uint4 code[4], rot;  // rot: word lane & 7 of row lane >> 3
      float scale;         // lane l < 16: group l & 3 of row l >> 2
    } u0, u1;
    const int odd = (lane >> 2) & 1, wch = lane & 3;
    // of the tile that is loaded: its descriptor's slot, and what this warp needs of it
    int ring = 0, b = 0;
    bool more = false, first = true;
    uint32_t valid = 0;
    const uint8_t* rows = a.cache;  // dense: the first of the warp's
    auto fetch = [&](int t) {
      ring = t % kInfo;
      if (!wait(&info_full[ring], (t / kInfo) & 1)) return false;
      const TileInfo& x = infos[ring];
      more = !(x.flags & kEnd);
      first = (x.flags & kFirst) != 0;
      b = x.b;
      valid = x.mask[w >> 2] >> (8 * (w & 3));
      if constexpr (!SPARSE) rows = a.cache + x.at[w >> 1] + (w & 1) * 8 * kLatentRowFp8;
      return true;
    };
    auto load = [&](Unit& v, int h) {  // four of the warp's rows
      const uint32_t m = valid >> (4 * h);
      auto row_of = [&](int j) -> const uint8_t* {
        if constexpr (SPARSE) return a.cache + places[ring * kT + 8 * w + 4 * h + j];
        else return rows + (4 * h + j) * kLatentRowFp8;
      };
      v.scale = 1.f;
      v.rot = make_uint4(0, 0, 0, 0);
      if (lane < 16 && ((m >> (lane >> 2)) & 1u)) v.scale = ld_nc_f(row_of(lane >> 2) + 512 + (lane & 3) * 4);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v.code[j] = make_uint4(0, 0, 0, 0);
        if ((m >> j) & 1u) v.code[j] = ld_nc_v4(row_of(j) + lane * 16);
      }
      if ((m >> (lane >> 3)) & 1u) v.rot = ld_nc_v4(row_of(lane >> 3) + 528 + (lane & 7) * 16);
    };
    uint32_t tile = 0;
    int n = 0, qn = -1;  // qn: stage of the last Q that this warp has copied
    // widens one unit into the tile in stage n; once its registers are read,
    // `then` asks for what they hold next
    auto widen = [&](Unit& v, int h, auto&& then) {
#pragma unroll
      for (int j = 0; j < 4; ++j) use_now(v.code[j]);  // the unit has arrived
      use_now(v.rot);
      // all four rows at once, with nothing ordered in between: two warps a
      // scheduler leave it to one warp's independent instructions to fill it
      uint32_t o[4][8];
      float f[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) f[j] = __shfl_sync(0xffffffffu, v.scale, 4 * j + (lane >> 3));
#pragma unroll
      for (int j = 0; j < 4; ++j) e4m3x16_to_bf16x16(v.code[j], f[j], o[j]);
      const uint4 rot = v.rot;
      if (!then()) return false;
      if (h == 0 && !wait(&freed[n % kStages], ((n / kStages) & 1) ^ 1)) return false;
      const int r0 = 8 * w + 4 * h;
      st_shared_v4(tile + 8 * kSlab + sw128_offset(r0 + (lane >> 3), lane & 7), rot);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint4 lo = make_uint4(o[j][0], o[j][1], o[j][2], o[j][3]), hi = make_uint4(o[j][4], o[j][5], o[j][6], o[j][7]);
        const uint32_t dst = tile + (lane >> 2) * kSlab;
        st_shared_v4(dst + sw128_offset(r0 + j, 2 * wch + odd), odd ? hi : lo);
        st_shared_v4(dst + sw128_offset(r0 + j, 2 * wch + 1 - odd), odd ? lo : hi);
      }
      return true;
    };
    bool ok = fetch(0);
    if (ok && more) {
      load(u0, 0);
      load(u1, 1);
      warp_arrive(&info_free[ring]);
    }
#pragma unroll 1
    for (int t = 0; ok && more; ++t) {
      // Every warp waits for every stage, Q's too, which the first of them
      // copies: a warp that skipped one could be two phases ahead at its next
      // wait, and take an older phase of the same parity for its own.
      if (kQStage && first) {
        const int qs = n % kStages;
        ok = wait(&freed[qs], ((n / kStages) & 1) ^ 1);
        if (!ok) break;
        if (w == 0) {
          if (lane == 0) {
            mbar_arrive_n(&full[qs], 7);
            mbar_arrive_expect_tx(&full[qs], 9 * R::kQSlab);
          }
          __syncwarp();
          copy_q(b, smem + qs * kTile, &full[qs]);
          qn = n;
        }
        ++n;
      }
      tile = smem_u32(smem) + (n % kStages) * kTile;
      ok = widen(u0, 0, [&] {
        if (!fetch(t + 1)) return false;
        if (more) load(u0, 0);
        return true;
      });
      if (!ok) break;
      ok = widen(u1, 1, [&] {
        if (more) {
          load(u1, 1);
          warp_arrive(&info_free[ring]);
        }
        return true;
      });
      if (!ok) break;
      fence_proxy_async_smem();
      warp_arrive(&full[n % kStages]);
      ++n;
    }
    // given up: the copy lands before the CTA exits (else the piece's products have waited for it)
    if (!ok && qn >= 0 && lane == 0) mbar_drain(&full[qn % kStages], (qn / kStages) & 1);
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the pieces of each sequence that more than one group worked on, and
// writes the rows of sequences without a tile. A warp has 32 query rows, one a
// lane, and 16 output dims; its reads of the partials, [dim / 4][row][4], are
// 512 bytes in a row. WPP warps share the pieces of one such part, each with its
// own running reference.
constexpr int kJoinThreads = 256;
template <bool SPARSE, int M, int WPP>
__global__ void __launch_bounds__(kJoinThreads) latent_join_kernel(const LatentArgs a) {
  constexpr int kPerCta = 8 / WPP;       // parts of a CTA
  constexpr int kCtas = 32 / kPerCta;    // CTAs of 32 rows
  __shared__ int64_t sums[2][8];
  __shared__ float4 accs[WPP > 1 ? 8 : 1][4][32];
  __shared__ float2 mls[WPP > 1 ? 8 : 1][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row32 = (a.rows + 31) / 32;
  const int b = blockIdx.x / (row32 * kCtas), rest = blockIdx.x - b * row32 * kCtas;
  const int row = rest / kCtas * 32 + lane;
  const int dim = (rest % kCtas * kPerCta + warp / WPP) * 16;
  pdl_trigger();
  // tiles of all sequences, and of those before b. (The lengths, the gate and the
  // sink were there before the main kernel started, which had no early start, so
  // they are read before it ends.)
  int64_t total = 0, start = 0;
  int bt;
  if (SPARSE) {
    bt = tiles_of(a.k);
    total = static_cast<int64_t>(a.B) * bt;
    start = static_cast<int64_t>(b) * bt;
  } else {
    bt = tiles_of(seq_len<SPARSE>(a, b));
    for (int i = threadIdx.x; i < a.B; i += kJoinThreads) {
      const int n = tiles_of(seq_len<SPARSE>(a, i));
      total += n;
      if (i < b) start += n;
    }
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
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      total += sums[0][i];
      start += sums[1][i];
    }
  }
  int gf = 0, gl = -1, first_slot = 0;
  const int G = eff_groups(a.groups, total);
  if (bt > 0) {
    // the group of the first tile, and of the last
    if (total < (1 << 22) && G < 512) {
      gf = static_cast<int>((static_cast<uint32_t>(start + 1) * static_cast<uint32_t>(G) - 1) / static_cast<uint32_t>(total));
      gl = static_cast<int>((static_cast<uint32_t>(start + bt) * static_cast<uint32_t>(G) - 1) / static_cast<uint32_t>(total));
    } else {
      gf = static_cast<int>(((start + 1) * G - 1) / total);
      gl = static_cast<int>(((start + bt) * G - 1) / total);
    }
    if (gf == gl) {  // one piece: written already
      pdl_wait();    // (no CTA ends before the main kernel, so that the stream's next one cannot start before it)
      return;
    }
    // only the first of the groups may hold another sequence before this one
    first_slot = share_start(gf, total, G) < start ? 1 : 0;
  }
  const bool live = row < a.rows;
  const int rb = row / M, r = row % M;
  const int64_t gr = static_cast<int64_t>(b) * a.rows + row;
  uint4 gates[2] = {};
  if (a.gate && live && warp % WPP == 0) {
    gates[0] = reinterpret_cast<const uint4*>(a.gate + gr * 512 + dim)[0];
    gates[1] = reinterpret_cast<const uint4*>(a.gate + gr * 512 + dim)[1];
  }
  const float sink2 = a.sink && live ? a.sink[row % a.H] * kLog2e : -INFINITY;
  pdl_wait();
  float m = -INFINITY, den = 0.f;
  float4 acc[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  if (live) {
#pragma unroll 4
    for (int g = gf + warp % WPP; g <= gl; g += WPP) {
      const int64_t block = static_cast<int64_t>(2 * g + (g == gf ? first_slot : 0)) * a.rblocks + rb;
      const float2 v = reinterpret_cast<const float2*>(a.part_ml)[block * M + r];
      const float4* src = reinterpret_cast<const float4*>(a.part_o) + (block * 128 + dim / 4) * M + r;
      const float4 p[4] = {src[0], src[M], src[2 * M], src[3 * M]};
      const float top = fmaxf(m, v.x);
      const float keep = m == -INFINITY ? 0.f : ex2_approx(m - top), w = v.x == -INFINITY ? 0.f : ex2_approx(v.x - top);
      m = top;
      den = fmaf(den, keep, w * v.y);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc[i].x = fmaf(acc[i].x, keep, w * p[i].x);
        acc[i].y = fmaf(acc[i].y, keep, w * p[i].y);
        acc[i].z = fmaf(acc[i].z, keep, w * p[i].z);
        acc[i].w = fmaf(acc[i].w, keep, w * p[i].w);
      }
    }
  }
  if constexpr (WPP > 1) {
#pragma unroll
    for (int i = 0; i < 4; ++i) accs[warp][i][lane] = acc[i];
    mls[warp][lane] = make_float2(m, den);
    __syncthreads();
    if (warp % WPP) return;
#pragma unroll 1
    for (int k = 1; k < WPP; ++k) {
      const float2 v = mls[warp + k][lane];
      const float top = fmaxf(m, v.x);
      const float keep = m == -INFINITY ? 0.f : ex2_approx(m - top), w = v.x == -INFINITY ? 0.f : ex2_approx(v.x - top);
      m = top;
      den = fmaf(den, keep, w * v.y);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 p = accs[warp + k][i][lane];
        acc[i].x = fmaf(acc[i].x, keep, w * p.x);
        acc[i].y = fmaf(acc[i].y, keep, w * p.y);
        acc[i].z = fmaf(acc[i].z, keep, w * p.z);
        acc[i].w = fmaf(acc[i].w, keep, w * p.w);
      }
    }
  }
  if (!live) return;
  const float top = fmaxf(m, sink2);
  const float w = m == -INFINITY ? 0.f : exp2f(m - top);
  den = den * w + (sink2 == -INFINITY ? 0.f : exp2f(sink2 - top));
  const float f = w > 0.f ? w / den : 0.f;
  float o[16];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    o[4 * i] = acc[i].x * f;
    o[4 * i + 1] = acc[i].y * f;
    o[4 * i + 2] = acc[i].z * f;
    o[4 * i + 3] = acc[i].w * f;
  }
  if (a.gate) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint32_t gw[4] = {gates[k].x, gates[k].y, gates[k].z, gates[k].w};
#pragma unroll
      for (int e = 0; e < 8; ++e)
        o[8 * k + e] *= __fdividef(1.f, 1.f + ex2_approx(-kLog2e * bf16_lane(gw[e >> 1], e & 1)));
    }
  }
  if (a.out_f32) {
    float4* dst = reinterpret_cast<float4*>(static_cast<float*>(a.out) + gr * 512 + dim);
#pragma unroll
    for (int i = 0; i < 4; ++i) dst[i] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
  } else {
    uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + gr * 512 + dim);
#pragma unroll
    for (int k = 0; k < 2; ++k)
      dst[k] = make_uint4(pack_bf16x2(o[8 * k], o[8 * k + 1]), pack_bf16x2(o[8 * k + 2], o[8 * k + 3]),
                          pack_bf16x2(o[8 * k + 4], o[8 * k + 5]), pack_bf16x2(o[8 * k + 6], o[8 * k + 7]));
  }
  if (a.lse && dim == 0) a.lse[gr] = top == -INFINITY ? -INFINITY : (top + log2f(den)) / kLog2e;
}

template <bool FP8, bool SPARSE, int M>
cudaError_t launch_one(const CUtensorMap& qmap, const CUtensorMap& kvmap, const LatentArgs& a, cudaStream_t stream) {
  using C = Cfg<FP8, SPARSE, M>;
  auto kern = latent_attention_kernel<FP8, SPARSE, M>;
  static bool done[64] = {false};
  const cudaError_t e = set_smem_once(kern, C::kSmemBytes, done);
  if (e != cudaSuccess) return e;
  // no early start here: the joining kernel, which has it, reads the call's inputs
  // before this one ends, and they are complete only because this one waited for
  // everything before it
  return launch_kernel(kern, dim3(static_cast<unsigned>(a.groups) * a.rblocks), dim3(C::kThreads), C::kSmemBytes, stream,
                       false, qmap, kvmap, a);
}

template <bool SPARSE, int M>
cudaError_t launch_join(const LatentArgs& a, cudaStream_t stream) {
  // Pieces of a sequence: about groups / B + 1. More than four are shared by eight
  // warps. us a call of B sequences of e4m3 rows, 131072 in all, by one warp / eight:
  //   B (pieces)    4        12       18       25       32       48
  //   8 heads    68/31    41/33    42/39    39/38    39/41    37/44   (38, 13, 9, 6, 5, 4 pieces)
  //   128 heads  67/45    55/60    60/71    57/74    63/82    62/95   (19, 7, 5, 3, 3, 2 pieces)
  // With 128 heads, where eight warps are four times as many CTAs of a grid that is
  // full already, the bound is 4 to 11 us on the wrong side at five to seven pieces.
  const bool many = a.groups / a.B + 1 > 4;
  const unsigned ctas = static_cast<unsigned>(a.B) * ((a.rows + 31) / 32) * (many ? 32 : 4);
  auto join = many ? latent_join_kernel<SPARSE, M, 8> : latent_join_kernel<SPARSE, M, 1>;
  return launch_kernel(join, dim3(ctas), dim3(kJoinThreads), 0, stream, true, a);
}

}  // namespace

cudaError_t launch_latent_attention(const CUtensorMap& qmap, const CUtensorMap& kvmap, const LatentArgs& a, bool fp8,
                                    bool sparse, cudaStream_t stream, int* launches) {
  const bool m32 = a.block == 32;
  cudaError_t e;
  if (latent_pair(a.rows))
    e = launch_latent_pair(qmap, kvmap, a, fp8, sparse, stream);
  else if (sparse)
    e = m32 ? launch_one<true, true, 32>(qmap, kvmap, a, stream) : launch_one<true, true, 64>(qmap, kvmap, a, stream);
  else if (fp8)
    e = m32 ? launch_one<true, false, 32>(qmap, kvmap, a, stream) : launch_one<true, false, 64>(qmap, kvmap, a, stream);
  else
    e = m32 ? launch_one<false, false, 32>(qmap, kvmap, a, stream) : launch_one<false, false, 64>(qmap, kvmap, a, stream);
  if (e != cudaSuccess) return e;
  e = sparse ? (m32 ? launch_join<true, 32>(a, stream) : launch_join<true, 64>(a, stream))
             : (m32 ? launch_join<false, 32>(a, stream) : launch_join<false, 64>(a, stream));
  if (e == cudaSuccess) *launches += 2;
  return e;
}

}  // namespace ic
