// Latent attention with a pair of CTAs for each block of 128 query rows (the
// mathematics, the split into shares and the joining are those of
// latent_attention.cu).
//
// Why a pair. The MMAs of one CTA read their operands from its shared memory at
// 128 bytes a cycle: 64 query rows against 64 keys cost 32 cycles a product of
// 16 dims, twice what the tensor core needs. A pair's MMA (cta_group::2, M =
// 128) has 64 rows in each CTA and takes half of the other operand from each, so
// it reads 3 KB where the single CTA reads 4, and 6 KB where it reads 10 (25 and
// 64 cycles, measured, against 32 and 80). And the two halves differ: for the
// logits CTA r holds its 32 keys of the tile with all their dims, for the output
// all 64 keys with its 256 dims. Keys and values then come and go by
// themselves, 36 and 32 KB each, where the single CTA holds 72 KB from the first
// product to the last and has room for two tiles in that state.
//
//   S[128 x 64]    = Q . K^T   (36 MMAs, N = 64: columns 32 r + [0, 32) are CTA r's keys)
//   O[128 x 512]  += P . V     (8 MMAs, N = 256: 128 dims of each CTA)
//
// In each CTA lanes 0-63 of TMEM hold its 64 rows' first half of the columns,
// lanes 64-127 the second, as in the single CTA's form.
//
// What bounds it. 32 ragged sequences of up to 8192 rows x 128 heads: 97 us a call
// from bf16 pages, 103 from e4m3, with inputs that change from call to call (87 and
// 100 in a graph; 9 of them joining), where HBM would take 35 and 21 and the MMAs
// 32. In the steady state a tile's MMAs take 1250 cycles, its chain of softmax
// (logits read, maxima exchanged between the halves, 2^x, weights stored and told to
// the first CTA) and products 2300 (e4m3: 2700), and the next tile's logits are all
// that runs beside it. Starts and pieces come on top (2970 cycles a tile on average,
// bf16): a share has 40 or 41 tiles in one to three pieces, and a further piece costs
// 12500 cycles, as much as five tiles, since the pair drains at its end (the next Q
// is copied after the last logits, the next product waits until the output has been
// read out and written). The one share of three pieces ends 11 us after the average.
// One buffer of weights: P(t) waits for the product of t - 1. A second (8 KB) would
// fit in the 9 KB that are free; for bf16 pages the registers of a second softmax
// warpgroup would be there too.
//
// Roles in each CTA. Warp 0 finds the tiles; warps 4-7 run the softmax and the
// output; a warp loads Q. In the first CTA warps 1 and 2 issue the products of
// both; what they wait for (Q, keys, values, weights) is told to its barriers by
// both CTAs, and their commits tell both. bf16 pages: warp 3 copies, warp 8 sees
// the copies land, clears the rows behind a sequence's end and passes the tile
// on. e4m3 pages: warps 8-15 widen their CTA's 32 keys, and the other's for its
// own 256 dims.
#include "latent.cuh"

namespace ic {

namespace {

constexpr int kKBytes = 9 * 4096;  // 32 rows of 576 dims: slabs of 32 rows x 64 dims
constexpr int kVBytes = 4 * kSlab;  // 64 rows of 256 dims
constexpr int kRows = 64;          // query rows of a CTA
using R64 = Rows<64>;

template <bool FP8, bool SPARSE>
struct PairCfg {
  static constexpr int kThreads = FP8 ? 512 : 320;
  static constexpr int kInfo = SPARSE ? 3 : 8;
  static constexpr int kOffK = 0;                       // [2]
  static constexpr int kOffV = 2 * 9 * 4096;            // [2]
  static constexpr int kOffQ = kOffV + 2 * 4 * kSlab;
  static constexpr int kOffP = kOffQ + 9 * R64::kQSlab;
  static constexpr int kOffX = kOffP + R64::kP;
  static constexpr int kOffInfo = kOffX + 2 * 128 * 4;
  static constexpr int kOffSlots = kOffInfo + kInfo * static_cast<int>(sizeof(TileInfo));
  static constexpr int kOffBar = kOffSlots + (SPARSE ? kInfo * kT * 8 : 0);
  // readers of a descriptor: warps 1 and 2, four softmax warps, the warp that
  // loads Q, and the copying and the passing warp or the widening warps
  static constexpr int kReaders = 7 + (FP8 ? 8 : 2);
  static constexpr int kNumBars = 2 * kInfo + 21;
  static constexpr int kOffMisc = kOffBar + kNumBars * 8;
  static constexpr int kSmemBytes = kOffMisc + 16;
  static_assert(kOffV % 1024 == 0 && kOffQ % 1024 == 0 && kOffP % 1024 == 0 && kOffBar % 8 == 0, "alignment");
  static_assert(kSmemBytes <= 232448, "fits one CTA per SM");
};

// ---------------------------------------------------------------- pair forms
IC_DEV void tmem_alloc_pair(uint32_t* holder, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(holder)), "r"(ncols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
IC_DEV void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
IC_DEV void mma_pair_bf16_ss(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Arrive on `bar` of both CTAs when every MMA issued so far by this thread has completed.
IC_DEV void commit_both(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_u32(bar)),
      "h"(static_cast<uint16_t>(3))
      : "memory");
}
IC_DEV void commit_pair(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}
// Arrive on a barrier of either CTA. What it tells of lies in this CTA's own shared
// memory or TMEM, where the pair's MMA reads it through the async proxy: copies
// that have landed and been waited for, stores that fence.proxy.async has made
// visible to that proxy before the arrival is issued, TMEM reads that have ended.
// PTX orders an arrival of this form for the threads of its own CTA; that the
// products which the first CTA issues after its wait find the second CTA's memory
// as its fences left it is relied on. Release and acquire at cluster scope would
// have the memory model say so: 1000 cycles an arrival, and the three batches of
// 128 heads take 121, 137 and 63 us then, 90, 103 and 53 now (inputs in turn).
IC_DEV void arrive_cluster(uint32_t addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}

template <bool FP8, bool SPARSE>
__global__ void __launch_bounds__(PairCfg<FP8, SPARSE>::kThreads, 1)
    latent_pair_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kvmap,
                       const LatentArgs a) {
  using C = PairCfg<FP8, SPARSE>;
  constexpr int kInfo = C::kInfo;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* ks = smem + C::kOffK;
  uint8_t* vs = smem + C::kOffV;
  uint8_t* qs = smem + C::kOffQ;
  uint8_t* ps = smem + C::kOffP;
  float* xm = reinterpret_cast<float*>(smem + C::kOffX);
  TileInfo* infos = reinterpret_cast<TileInfo*>(smem + C::kOffInfo);
  int64_t* places = reinterpret_cast<int64_t*>(smem + C::kOffSlots);
  uint64_t* info_full = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  uint64_t* info_free = info_full + kInfo;
  // in each CTA
  uint64_t* s_full = info_free + kInfo;  // [2] a tile's logits are in TMEM, and its keys have been read
  uint64_t* pv_done = s_full + 2;        // [2] its values and weights have been read
  uint64_t* q_free = pv_done + 2;        // the piece's last logits have been formed
  uint64_t* xch = q_free + 1;            // [2] the softmax warps that share rows exchange a value
  uint64_t* k_landed = xch + 2;          // [2] bf16: copies
  uint64_t* v_landed = k_landed + 2;     // [2]
  uint64_t* q_landed = v_landed + 2;
  // in the first CTA, told by both
  uint64_t* q_full = q_landed + 1;
  uint64_t* k_full = q_full + 1;         // [2]
  uint64_t* v_full = k_full + 2;         // [2]
  uint64_t* p_ready = v_full + 2;        // [2] weights of a tile in shared memory, its logits read, O rescaled
  uint64_t* o_free = p_ready + 2;        // a piece's output has been read out
  uint64_t* retire = o_free + 1;         // (21 in all, from s_full)
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 4);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  const int pairs = a.rblocks >> 1;  // blocks of 128 rows
  const int cluster = blockIdx.x >> 1;
  const int group = cluster / pairs, rb = 2 * (cluster - group * pairs) + rank;  // rb: block of 64 rows
  pdl_trigger();
  if (threadIdx.x == 0) {
    tma_prefetch_desc(&qmap);
    if (!FP8) tma_prefetch_desc(&kvmap);
    for (int i = 0; i < kInfo; ++i) {
      mbar_init(&info_full[i], 1);
      mbar_init(&info_free[i], C::kReaders);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&pv_done[i], 1);
      mbar_init(&xch[i], 2);
      mbar_init(&k_landed[i], 1);
      mbar_init(&v_landed[i], 1);
      mbar_init(&k_full[i], FP8 ? 16 : 2);
      mbar_init(&v_full[i], FP8 ? 16 : 2);
      mbar_init(&p_ready[i], 8);
    }
    mbar_init(q_free, 1);
    mbar_init(q_landed, 1);
    mbar_init(q_full, 2);
    mbar_init(o_free, 8);
    mbar_init(retire, 2);
    *abort_flag = 0;
    fence_mbar_init();
  }
  pdl_wait();
  const int64_t len0 = !SPARSE && warp == 0 && lane < a.B ? a.lens[lane] : 0;
  // the swizzled layouts need a 1024-byte-aligned base (the same in both CTAs)
  const bool aligned = (smem_u32(smem) & 1023u) == 0;
  if (!aligned && threadIdx.x == 0) record_status(a.status, IC_ERR_UNSUPPORTED);
  if (warp == 1) tmem_alloc_pair(tmem_holder, 512);
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // the barriers of both CTAs are there
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait_hot(bar, parity, abort_flag, a.status, a.wait_ns)) != 0;
  };
  auto warp_arrive = [&](uint64_t* bar) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
    __syncwarp();
  };
  // on a barrier of the first CTA
  auto tell_first = [&](uint64_t* bar) {
    __syncwarp();
    if (lane == 0) arrive_cluster(dsmem_addr(bar, 0));
    __syncwarp();
  };
  auto get_info = [&](int t, TileInfo& x) {
    if (!wait(&info_full[t % kInfo], (t / kInfo) & 1)) return false;
    x = infos[t % kInfo];
    warp_arrive(&info_free[t % kInfo]);
    return true;
  };
  const int br = a.page_size % 32 == 0 ? 32 : 16;  // rows of a TMA box

  auto load_q = [&] {
    // ------------------------------------------------------------ Q of each piece
    int pieces = 0;
    for (int t = 0;; ++t) {
      TileInfo x;
      if (!get_info(t, x) || (x.flags & kEnd)) break;
      if (!(x.flags & kFirst)) continue;
      if (pieces > 0 && !wait(q_free, (pieces - 1) & 1)) break;
      if (elect_one()) {
        mbar_arrive_expect_tx(q_landed, 9 * R64::kQSlab);
        // rows of the next sequence, or zeros, behind this one's: not written out
#pragma unroll
        for (int c = 0; c < 9; ++c)
          tma_load_2d(qs + c * R64::kQSlab, &qmap, q_landed, c * 64, x.b * a.rows + rb * kRows);
      }
      __syncwarp();
      ++pieces;
      if (!wait(q_landed, (pieces - 1) & 1)) break;
      tell_first(q_full);
    }
    if (pieces > 0) mbar_drain(q_landed, (pieces - 1) & 1);
  };

  if (!aligned) {
    // (nothing runs)
  } else if (warp < 4) {
    // (one branch for each four warps, as in the single CTA's kernel: fewer registers)
    if (warp == 0) {
      find_tiles<FP8, SPARSE, kInfo>(a, len0, group, 16, rank, infos, places, info_full, info_free, wait);
    } else if (warp == 1) {
      // ------------------------------------------------------------ S = Q . K^T
      constexpr uint32_t idesc = idesc_bf16_f32(128, kT, false, false);
      int pieces = 0;
#pragma unroll 1
      for (int t = 0;; ++t) {
        TileInfo x;
        if (!get_info(t, x) || (x.flags & kEnd)) break;
        if (rank != 0) continue;
        if (x.flags & kFirst) {
          if (!wait(q_full, pieces & 1)) break;
          ++pieces;
        }
        // the logits of tile t - 2 have been read
        if (t >= 2 && !wait(&p_ready[t & 1], ((t >> 1) - 1) & 1)) break;
        if (!wait(&k_full[t & 1], (t >> 1) & 1)) break;
        tc_fence_after();
        if (elect_one()) {
          const uint32_t d = tmem + R64::kSCol + (t & 1) * R64::kCols;
          const uint64_t ad = sw128_desc(smem_u32(qs), 16, 1024), bd = sw128_desc(smem_u32(ks) + (t & 1) * kKBytes, 16, 1024);
#pragma unroll 1
          for (int c = 0; c < 9; ++c)
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_pair_bf16_ss(d, ad + c * (R64::kQSlab >> 4) + kk * 2, bd + c * (4096 >> 4) + kk * 2, idesc, c + kk > 0);
          commit_both(&s_full[t & 1]);
          if (x.flags & kLast) commit_both(q_free);
        }
        __syncwarp();
      }
      // every MMA issued has retired before TMEM is released
      if (rank == 0) {
        if (elect_one()) commit_pair(retire);
        __syncwarp();
        mbar_drain(retire, 0);
      }
    } else if (warp == 2) {
      // ------------------------------------------------------------ O += P . V
      constexpr uint32_t idesc = idesc_bf16_f32(128, 256, false, true);
      int pieces = 0;
#pragma unroll 1
      for (int t = 0;; ++t) {
        TileInfo x;
        if (!get_info(t, x) || (x.flags & kEnd)) break;
        if (rank != 0) continue;
        const bool first = (x.flags & kFirst) != 0;
        if (first) {
          if (pieces > 0 && !wait(o_free, (pieces - 1) & 1)) break;
          ++pieces;
        }
        if (!wait(&v_full[t & 1], (t >> 1) & 1)) break;
        if (!wait(&p_ready[t & 1], (t >> 1) & 1)) break;
        tc_fence_after();
        if (elect_one()) {
          const uint64_t vd = sw128_desc(smem_u32(vs) + (t & 1) * kVBytes, kSlab, 1024), pd = sw128_desc(smem_u32(ps), 16, 1024);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
#pragma unroll
            for (int h = 0; h < 2; ++h)
              mma_pair_bf16_ss(tmem + R64::kOutCol + h * 128, pd + kk * 2, vd + h * (2 * kSlab >> 4) + kk * 128, idesc,
                               !first || kk > 0);
          commit_both(&pv_done[t & 1]);
        }
        __syncwarp();
      }
      if (rank == 0) {
        if (elect_one()) commit_pair(retire);
        __syncwarp();
        mbar_drain(retire, 0);
      }
    } else if (!FP8 && warp == 3) {
      // ------------------------------------------------------------ copies (bf16)
      int nk = 0, nv = 0;
      for (int t = 0;; ++t) {
        TileInfo x;
        if (!get_info(t, x) || (x.flags & kEnd)) break;
        // boxes without a valid row read the page behind the last, which fills zeros
        auto copy = [&](uint8_t* dst, uint64_t* bar, int i, int col) {  // 16 rows (or 32) from unit i on
          const int pz = x.at[i] < 0 ? a.num_pages : static_cast<int>(x.at[i]);
          tma_load_3d(dst, &kvmap, bar, col, (x.row0 + 16 * i) % a.page_size, pz);
        };
        const int ring = t & 1;
        if (t >= 2 && !wait(&s_full[ring], ((t >> 1) - 1) & 1)) break;
        if (elect_one()) {
          uint8_t* dst = ks + ring * kKBytes;
          mbar_arrive_expect_tx(&k_landed[ring], kKBytes);
#pragma unroll 1
          for (int c = 0; c < 9; ++c) {
            copy(dst + c * 4096, &k_landed[ring], 2 * rank, c * 64);
            if (br == 16) copy(dst + c * 4096 + 2048, &k_landed[ring], 2 * rank + 1, c * 64);
          }
        }
        __syncwarp();
        ++nk;
        if (t >= 2 && !wait(&pv_done[ring], ((t >> 1) - 1) & 1)) break;
        if (elect_one()) {
          uint8_t* dst = vs + ring * kVBytes;
          mbar_arrive_expect_tx(&v_landed[ring], kVBytes);
#pragma unroll 1
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (br == 16 || (i & 1) == 0) copy(dst + c * kSlab + i * 2048, &v_landed[ring], i, rank * 256 + c * 64);
        }
        __syncwarp();
        ++nv;
      }
      // the last copies land before the CTA exits, whatever their readers do
      for (int u = nk > 2 ? nk - 2 : 0; u < nk; ++u) mbar_drain(&k_landed[u & 1], (u >> 1) & 1);
      for (int u = nv > 2 ? nv - 2 : 0; u < nv; ++u) mbar_drain(&v_landed[u & 1], (u >> 1) & 1);
    } else {
      load_q();
    }
  } else if (warp < 8) {
    // ------------------------------------------------------------ softmax and output
    softmax_rows<64, true>(a, tmem, ps, xm, s_full, pv_done, q_free, xch, rb * kRows, rb, wait, warp_arrive, get_info,
                           [](uint32_t) { return true; }, [&](int t) { tell_first(&p_ready[t & 1]); },
                           [&]() { tell_first(o_free); });
  } else if (!FP8 && warp == 9) {
    load_q();
  } else if (!FP8) {
    // ------------------------------------------------------------ tiles passed on (bf16)
    for (int t = 0;; ++t) {
      TileInfo x;
      if (!get_info(t, x) || (x.flags & kEnd)) break;
      const int ring = t & 1;
      if (!wait(&k_landed[ring], (t >> 1) & 1)) break;
      tell_first(&k_full[ring]);
      if (!wait(&v_landed[ring], (t >> 1) & 1)) break;
      if (x.flags & kClear) {  // rows that hold nothing: a zero weight times a NaN left there would be NaN
        const uint32_t base = smem_u32(vs) + ring * kVBytes + (lane >> 3) * kSlab + (lane & 7) * 16;
#pragma unroll 8
        for (int r = 0; r < kT; ++r)
          if (!(((r & 32 ? x.mask[1] : x.mask[0]) >> (r & 31)) & 1u)) st_shared_v4(base + r * 128, make_uint4(0, 0, 0, 0));
        fence_proxy_async_smem();
      }
      tell_first(&v_full[ring]);
    }
  } else {
    // ------------------------------------------------------------ widening (e4m3)
    // Warp w has four of this CTA's 32 keys of the tile: a load takes a whole
    // row's codes, lane l the 16 of word l, and they are stored as keys, and those
    // of this CTA's 256 output dims as values too. The same four of the other
    // CTA's keys are read for those dims alone, two rows a load. (Sent across the
    // pair instead, they cost a fence and a release at cluster scope, 2000 cycles a
    // tile against 300 for widening them here.) Eight lanes that store together
    // have four words of two neighbouring slabs; those of the odd slab store their
    // second half first, so the eight meet eight chunks of the swizzle. The next
    // tile's loads are issued as soon as this one's codes are converted: a second
    // set of codes' registers would be spilled.
    const int w = warp - 8;
    struct Unit {
      uint4 code[4], rot;   // rot: word lane & 7 of row lane >> 3
      uint4 far[2];         // word lane & 15 of this CTA's dims of the other CTA's row 2 i + (lane >> 4)
      float scale;          // lane l < 16: group l & 3 of row l >> 2
      float far_scale;      // lane l < 8: group 2 rank + (l & 1) of the other CTA's row l >> 1
    } u;
    const int odd = (lane >> 2) & 1, wch = lane & 3;
    const int r0 = 4 * w;  // first of the warp's rows among the 32
    const uint32_t vto = smem_u32(vs) + ((lane >> 2) & 3) * kSlab;
    const uint32_t kto = smem_u32(ks) + (lane >> 2) * 4096;
    const bool mine = (lane >> 4) == rank;  // this lane's word of an own row is of this CTA's dims
    bool more = false;
    auto fetch = [&](int t) {  // tile t's descriptor, and its words on their way
      const int ring = t % kInfo;
      if (!wait(&info_full[ring], (t / kInfo) & 1)) return false;
      const TileInfo& x = infos[ring];
      more = !(x.flags & kEnd);
      if (more) {
        const uint32_t m = x.mask[rank] >> r0, mf = x.mask[1 - rank] >> r0;
        const uint8_t *base = a.cache, *fbase = a.cache;  // dense: the first of the four rows
        if constexpr (!SPARSE) {
          base += x.at[2 * rank + (w >> 2)] + (r0 & 15) * kLatentRowFp8;
          fbase += x.at[2 - 2 * rank + (w >> 2)] + (r0 & 15) * kLatentRowFp8;
        }
        auto row_of = [&](int j) -> const uint8_t* {
          if constexpr (SPARSE) return a.cache + places[ring * kT + 32 * rank + r0 + j];
          else return base + j * kLatentRowFp8;
        };
        auto far_of = [&](int j) -> const uint8_t* {
          if constexpr (SPARSE) return a.cache + places[ring * kT + 32 - 32 * rank + r0 + j];
          else return fbase + j * kLatentRowFp8;
        };
        u.scale = u.far_scale = 1.f;
        u.rot = make_uint4(0, 0, 0, 0);
        if (lane < 16 && ((m >> (lane >> 2)) & 1u)) u.scale = ld_nc_f(row_of(lane >> 2) + 512 + (lane & 3) * 4);
        if (lane < 8 && ((mf >> (lane >> 1)) & 1u))
          u.far_scale = ld_nc_f(far_of(lane >> 1) + 512 + (2 * rank + (lane & 1)) * 4);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          u.code[j] = make_uint4(0, 0, 0, 0);
          if ((m >> j) & 1u) u.code[j] = ld_nc_v4(row_of(j) + lane * 16);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int j = 2 * i + (lane >> 4);
          u.far[i] = make_uint4(0, 0, 0, 0);
          if ((mf >> j) & 1u) u.far[i] = ld_nc_v4(far_of(j) + rank * 256 + (lane & 15) * 16);
        }
        if ((m >> (lane >> 3)) & 1u) u.rot = ld_nc_v4(row_of(lane >> 3) + 528 + (lane & 7) * 16);
      }
      warp_arrive(&info_free[ring]);
      return true;
    };
    bool ok = fetch(0);
#pragma unroll 1
    for (int t = 0; ok && more; ++t) {
      const int ring = t & 1;
#pragma unroll
      for (int j = 0; j < 4; ++j) use_now(u.code[j]);  // the tile's words have arrived
      use_now(u.far[0]);
      use_now(u.far[1]);
      use_now(u.rot);
      uint32_t o[4][8], of[2][8];
      float f[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) f[j] = __shfl_sync(0xffffffffu, u.scale, 4 * j + (lane >> 3));
#pragma unroll
      for (int j = 0; j < 4; ++j) e4m3x16_to_bf16x16(u.code[j], f[j], o[j]);
#pragma unroll
      for (int i = 0; i < 2; ++i)
        e4m3x16_to_bf16x16(u.far[i], __shfl_sync(0xffffffffu, u.far_scale, 2 * (2 * i + (lane >> 4)) + ((lane >> 3) & 1)),
                           of[i]);
      const uint4 rot = u.rot;
      ok = fetch(t + 1);
      if (!ok) break;
      if (t >= 2) {
        ok = wait(&s_full[ring], ((t >> 1) - 1) & 1);  // the keys of tile t - 2 have been read
        if (!ok) break;
      }
      st_shared_v4(smem_u32(ks) + ring * kKBytes + 8 * 4096 + sw128_offset(r0 + (lane >> 3), lane & 7), rot);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint4 lo = make_uint4(o[j][0], o[j][1], o[j][2], o[j][3]), hi = make_uint4(o[j][4], o[j][5], o[j][6], o[j][7]);
        const uint32_t dst = kto + ring * kKBytes;
        st_shared_v4(dst + sw128_offset(r0 + j, 2 * wch + odd), odd ? hi : lo);
        st_shared_v4(dst + sw128_offset(r0 + j, 2 * wch + 1 - odd), odd ? lo : hi);
      }
      fence_proxy_async_smem();
      tell_first(&k_full[ring]);
      if (t >= 2) {
        ok = wait(&pv_done[ring], ((t >> 1) - 1) & 1);  // and its values
        if (!ok) break;
      }
      const uint32_t dst = vto + ring * kVBytes;
      if (mine) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint4 lo = make_uint4(o[j][0], o[j][1], o[j][2], o[j][3]), hi = make_uint4(o[j][4], o[j][5], o[j][6], o[j][7]);
          st_shared_v4(dst + sw128_offset(32 * rank + r0 + j, 2 * wch + odd), odd ? hi : lo);
          st_shared_v4(dst + sw128_offset(32 * rank + r0 + j, 2 * wch + 1 - odd), odd ? lo : hi);
        }
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int j = 2 * i + (lane >> 4);
        const uint4 lo = make_uint4(of[i][0], of[i][1], of[i][2], of[i][3]), hi = make_uint4(of[i][4], of[i][5], of[i][6], of[i][7]);
        const int row = 32 - 32 * rank + r0 + j;
        st_shared_v4(dst + sw128_offset(row, 2 * wch + odd), odd ? hi : lo);
        st_shared_v4(dst + sw128_offset(row, 2 * wch + 1 - odd), odd ? lo : hi);
      }
      fence_proxy_async_smem();
      tell_first(&v_full[ring]);
    }
  }

  // neither CTA leaves before the other has done with its memory (every wait
  // above ends by itself)
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

template <bool FP8, bool SPARSE>
cudaError_t launch_pair(const CUtensorMap& qmap, const CUtensorMap& kvmap, const LatentArgs& a, cudaStream_t stream) {
  using C = PairCfg<FP8, SPARSE>;
  auto kern = latent_pair_kernel<FP8, SPARSE>;
  static bool done[64] = {false};
  const cudaError_t e = set_smem_once(kern, C::kSmemBytes, done);
  if (e != cudaSuccess) return e;
  // no early start: the joining kernel relies on it (launch_one in latent_attention.cu)
  return launch_kernel_cluster(kern, dim3(static_cast<unsigned>(a.groups) * a.rblocks), dim3(C::kThreads), C::kSmemBytes,
                               stream, false, 2, qmap, kvmap, a);
}

}  // namespace

cudaError_t launch_latent_pair(const CUtensorMap& qmap, const CUtensorMap& kvmap, const LatentArgs& a, bool fp8,
                               bool sparse, cudaStream_t stream) {
  return sparse ? launch_pair<true, true>(qmap, kvmap, a, stream)
         : fp8  ? launch_pair<true, false>(qmap, kvmap, a, stream)
                : launch_pair<false, false>(qmap, kvmap, a, stream);
}

}  // namespace ic
