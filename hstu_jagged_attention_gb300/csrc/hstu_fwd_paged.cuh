// The attention of many new tokens over the paged cache, on tcgen05: the
// roles and the TMEM layout of the forward kernel (hstu_fwd.cu), with
//   - K and V blocks of 128 keys gathered page by page (one bulk-tensor copy
//     a page and 64-channel chunk);
//   - tiles of 128 new tokens at any position: the keys a row may see end
//     anywhere in a block, and candidates see the history and themselves;
//   - equal shares of (tile, sequence, head, key block) units per CTA, so an
//     item may be cut between CTAs; its parts are summed in their order by
//     the CTA that arrives last.
// Bound by the same stages as the forward (SiLU on the MUFU and the issue
// slots, the split P's products; ncu: MUFU 47%, issue 55%, tensor pipe 37%
// busy): 1024 candidates of 32 users against 2048 to 8192 tokens, 4 heads of
// 64, take 289 us (167 GFLOP, 578 TF/s), 1.03 us a 128 x 128 block; at d = 128
// 1.6 to 1.8 us a block (chunks of 100 to 700 tokens: 70 us, 578 TF/s).
// Included by hstu_fwd.cu.

// What the K producer, which runs ahead of every other role, leaves in shared
// memory for them: a word per step (key block) and one per item.  Each role
// then follows the CTA's steps 0 .. n - 1 with no schedule of its own: with
// the cursor inlined in every role, the kernel missed the instruction cache
// (73.7% hits, 88% of the cache's fill bandwidth) and the candidates took 494
// us; with these words 357, and with the product issuers' loops not unrolled
// over the three buffers 318 (now 96.6% hits).
// A word is written before its step's K copy is armed, so a role that has
// waited for the step's barrier finds it.  When the word of step c is
// written, QK(c - 3) and so PV(c - 6) are done: 8 step words are enough.  An
// item is at most 6 steps ahead of the PV issuer, and that at most two items
// ahead of the epilogue: 16 item words are enough.  (The 4-bit form's words are
// written when the codes' copy is, up to four steps ahead of that, hence 16
// step words.)
constexpr int kStepWords = 16, kItemWords = 16;
constexpr int kPagedThreads = 768;  // four SiLU warpgroups, the wide P layout, at every d
// What the keys and values come from: the bf16 pools' tensor maps, or the pages
// of 4-bit codes, which two warps each turn into the bf16 tiles.  Those are the
// first four (the keys' on even, the values' on odd schedulers), and the
// epilogue the last: candidates 332 us, 340 with them the other way round.
struct PagedMaps {
  CUtensorMap k, v;
};
constexpr int kUnpackWarps = 2, kSiluWarps = 16;
template <class SRC>
constexpr bool kHeldInQ4 = std::is_same<SRC, Q4Pool>::value;
template <class SRC>
constexpr int kPagedThreadsOf = kPagedThreads + (kHeldInQ4<SRC> ? 2 * 32 * kUnpackWarps : 0);
struct PagedStep {
  int lim;    // position of the tile's first row, less the block's first key
  int hist;   // history end, less the block's first key
  int rows;   // valid rows
  int edge;   // bit 0: the item's first step, bit 1: its last
  // First key (of the block) that no row sees; may be past the block.
  __device__ __forceinline__ int end() const { return lim + rows; }
  // Keys of the block that some row sees, up to the MMA's steps of 16.
  __device__ __forceinline__ int cols() const {
    const int r = end();
    return r >= kBN ? kBN : ((r + 15) & ~15);
  }
  // Every row sees every key of the block.
  __device__ __forceinline__ bool plain() const { return lim >= kBN - 1 && hist >= kBN; }
  __device__ __forceinline__ bool first() const { return edge & 1; }
  __device__ __forceinline__ bool last() const { return edge & 2; }
};
struct PagedItem {
  int row0, h, rows, blocks, c0, parts;
};
struct PagedWords {
  int4 step[kStepWords];
  PagedItem item[kItemWords];
  // the items shared with earlier and with later CTAs (parts == 0: none), and
  // which of them this CTA sums
  PagedItem cut[2];
  unsigned last;
};
// CTA `cta`'s part of the item that an earlier CTA starts (0) or that it starts (1).
template <int D>
__device__ __forceinline__ float4* paged_part(const PagedFwdArgs& a, int cta, int starts) {
  return reinterpret_cast<float4*>(a.parts) + ((long long)cta * 2 + starts) * (kBM * D / 4);
}
__device__ __forceinline__ PagedStep read_step(const PagedWords* words, uint32_t tc) {
  PagedStep s;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(s.lim), "=r"(s.hist), "=r"(s.rows), "=r"(s.edge)
               : "r"(smem_u32(words->step + tc % kStepWords))
               : "memory");
  return s;
}

// As Cfg's, where the unpacking warps arrive for their part of a tile.
template <int D, bool Q4>
__device__ constexpr uint32_t paged_arrivals(int i) {
  using C = Cfg<D>;
  const bool k = i >= C::B_QKREADY && i < C::B_QKREADY + C::P, v = i >= C::B_VFULL && i < C::B_VFULL + C::P;
  return C::arrivals(i, true) + (Q4 && (k || v) ? kUnpackWarps - 1u : 0u);
}

// One warp: the K stream with each item's Q tile, or the V stream.
template <int D, bool KQ>
__device__ void paged_producer(const CUtensorMap* tm, const CUtensorMap* tm_q, const PagedFwdArgs& a,
                               const PagedWork& w, PagedCursor cur, PagedSeg g, PagedWords* words,
                               uint32_t base, const WaitCtx& wt) {
  using C = Cfg<D>;
  constexpr int FULL = KQ ? C::B_QKREADY : C::B_VFULL;
  constexpr int OFF = KQ ? C::K_OFF : C::V_OFF;
  const uint32_t bars = base + C::BAR_OFF;
  auto bar = [&](int i) { return bars + 8u * (uint32_t)i; };
  const int lane = threadIdx.x & 31;
  const int shift = a.p.page_shift, ps = 1 << shift;
  const int box = ps < kBN ? ps : kBN;
  uint32_t c = 0, qc = 0;
  bool ok = true;
  while (ok && cur.next(a.p, w, &g)) {
    if (KQ) {
      const int qs = (int)(qc % C::QS);
      if (!(ok = wait_warp(bar(C::B_QEMPTY + qs), ((qc / C::QS) & 1u) ^ 1u, wt, kSiteQEmpty))) break;
      if (lane == 0) {
        words->item[qc % kItemWords] =
            PagedItem{g.seq.q0 + kBM * g.qt, g.h, g.walk.rows, g.n, g.c0, g.parts};
        mbar_arrive_expect_tx(bar(C::B_QFULL + qs), C::TILEB);
#pragma unroll
        for (int ch = 0; ch < C::NCHUNK; ++ch)
          tma_load_3d(base + C::Q_OFF + qs * C::TILEB + ch * C::CHUNKB, tm_q, bar(C::B_QFULL + qs),
                      ch * C::CHUNK, g.h, g.seq.q0 + kBM * g.qt);
      }
      ++qc;
    }
    const int32_t* row = a.p.page_table + (long long)g.b * a.p.max_pages;
    const int end = g.walk.end();
    const int pages = (end + ps - 1) >> shift;
    PageIds ids;
    for (int i = 0; i < g.n; ++i) {
      const int tok0 = kBN * g.walk.block(g.i0 + i);
      const int p0 = tok0 >> shift;
      const int valid = end - tok0 < kBN ? end - tok0 : kBN;
      const int npg = ps >= kBN ? 1 : (valid + ps - 1) >> shift;
      ids.cover(row, p0, npg, pages);
      const int pg = lane / C::NCHUNK, ch = lane % C::NCHUNK;  // npg NCHUNK <= 16 lanes copy
      int page = ids.get(p0 + pg);
      const int slot = (int)(c % C::P);
      // no further K copies once the CTA has given up (see the PV issuer's end);
      // one lane asks: all of them, with a vote, took 291.8 us on the candidates, 288 so
      if (lane == 0)
        ok = KQ ? wait_one(bar(C::B_SFULL + slot), ((c / C::P) & 1u) ^ 1u, wt, kSiteKEmpty) && !*wt.abort_flag
                : wait_one(bar(C::B_QKREADY + slot), (c / C::P) & 1u, wt, kSiteVEmpty);
      ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
      if (!ok) break;
      if (lane == 0) {
        if (KQ)
          words->step[c % kStepWords] = make_int4(g.walk.p0 - tok0, g.seq.hist - tok0, g.walk.rows,
                                                  (i == 0 ? 1 : 0) | (i == g.n - 1 ? 2 : 0));
        mbar_arrive_expect_tx(bar(FULL + slot), (uint32_t)(npg * box * C::ROWB * C::NCHUNK));
      }
      __syncwarp();
      if (pg < npg) {
        if (page < 0 || page >= a.p.num_pages) {
          // read as zeros, past the pool's end: silu(0) V = 0
          atomicOr(&g_dev_words[0], kStatusBadPaged);
          page = a.p.num_pages;
        }
        tma_load_4d(base + OFF + slot * C::TILEB + ch * C::CHUNKB + pg * box * C::ROWB, tm,
                    bar(FULL + slot), ch * C::CHUNK, g.h, ps >= kBN ? (tok0 & (ps - 1)) : 0, page);
      }
      ++c;
    }
  }
  // every copy lands before the CTA ends, also where the roles that would wait
  // for it have given up
  if (lane == 0) {
    drain_copies(bar(FULL), C::P, c);
    if (KQ) drain_copies(bar(C::B_QFULL), C::QS, qc);
  }
  __syncwarp();
}

// Shared memory of the 4-bit form.  At d = 128 the tiles fill it, so the keys
// get two slots instead of three: key slot t mod KP is free once QK(t - KP) has
// completed.  In that third slot's place (at d <= 64 behind the barriers) are
// the rings of codes on their way: a stage holds the codes of 128 keys, or
// values, d / 2 bytes a row, and then their scales, d / 16 bytes a row.
template <int D, bool Q4>
struct PagedCfg {
  using C = Cfg<D>;
  static constexpr int KP = Q4 && D == 128 ? 2 : C::P;
  static constexpr int KSTAGES = D == 128 ? 2 : 4, VSTAGES = D == 128 ? 1 : 4;
  static constexpr int RAWB = kBN * (D / 2 + D / kQ4Group);
  static constexpr int RAW_OFF = D == 128 ? C::K_OFF + KP * C::TILEB : (C::MISC_OFF + 16 + 127) / 128 * 128;
  static constexpr int RAW_BARS = RAW_OFF + (KSTAGES + VSTAGES) * RAWB;  // full, then empty
  static constexpr int RAW_END = RAW_BARS + 16 * (KSTAGES + VSTAGES);
  static constexpr int SMEM = !Q4 || D == 128 || RAW_END + 1024 <= C::SMEM_LAUNCH ? C::SMEM_LAUNCH : RAW_END + 1024;
  static_assert(!Q4 || D != 128 || RAW_END <= C::V_OFF, "the codes on their way");
  static_assert(SMEM <= 232448, "shared memory budget");
};
// The ring of the keys' (which = 0) or the values' codes: stage s, its full and
// its empty barrier.
template <int D>
struct RawRing {
  using U = PagedCfg<D, true>;
  uint32_t base;
  int which;
  __device__ __forceinline__ int stages() const { return which ? U::VSTAGES : U::KSTAGES; }
  __device__ __forceinline__ uint32_t stage(int s) const {
    return base + U::RAW_OFF + (uint32_t)((which ? U::KSTAGES : 0) + s) * U::RAWB;
  }
  __device__ __forceinline__ uint32_t full(int s) const {
    return base + U::RAW_BARS + 8u * (uint32_t)((which ? U::KSTAGES : 0) + s);
  }
  __device__ __forceinline__ uint32_t empty(int s) const { return full(s) + 8u * (U::KSTAGES + U::VSTAGES); }
};

// The copies of a cache of 4-bit codes, one warp for the keys (which = 0, with
// the words of every step and item) and one for the values: as paged_producer,
// two bulk copies a page into the ring of codes.
template <int D>
__device__ void paged_copy_codes(const Q4Pool& pool, const PagedFwdArgs& a, const PagedWork& w, PagedCursor cur,
                                 PagedSeg g, PagedWords* words, uint32_t base, const WaitCtx& wt, int which) {
  using U = PagedCfg<D, true>;
  using T = Q4Tile<D>;
  const RawRing<D> ring{base, which};
  const int lane = threadIdx.x & 31;
  const int shift = a.p.page_shift, ps = 1 << shift, ts = pool.tile_shift;
  uint32_t c = 0, qc = 0, round = 0;
  int st = 0;
  bool ok = true;
  while (ok && cur.next(a.p, w, &g)) {
    if (which == 0 && lane == 0)
      words->item[qc % kItemWords] = PagedItem{g.seq.q0 + kBM * g.qt, g.h, g.walk.rows, g.n, g.c0, g.parts};
    ++qc;
    const int32_t* row = a.p.page_table + (long long)g.b * a.p.max_pages;
    const int end = g.walk.end();
    const int pages = (end + ps - 1) >> shift;
    PageIds ids;
    for (int i = 0; i < g.n; ++i) {
      const int tok0 = kBN * g.walk.block(g.i0 + i);
      const int p0 = tok0 >> shift;
      const int valid = end - tok0 < kBN ? end - tok0 : kBN;
      const int npg = ps >= kBN ? 1 : (valid + ps - 1) >> shift;  // at most 8
      ids.cover(row, p0, npg, pages);
      // lanes 0 .. npg - 1 copy codes, lanes 16 .. 16 + npg - 1 scales
      const int pg = lane & 15, part = lane >> 4;
      const int page = ids.get(p0 + pg);
      if (lane == 0)
        ok = wait_one(ring.empty(st), (round & 1u) ^ 1u, wt, which ? kSiteVEmpty : kSiteKEmpty) && !*wt.abort_flag;
      ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
      if (!ok) break;
      const bool mine = pg < npg, good = page >= 0 && page < a.p.num_pages;
      const unsigned bad = __ballot_sync(0xffffffffu, mine && !good);
      const int bytes = (part ? T::SCALEB : T::CODEB) << ts;
      const uint32_t dst = ring.stage(st) + (part ? kBN * T::CODEB : 0) + pg * bytes;
      if (bad) {
        if (mine && !good) {
          // read as zeros: silu(0) V = 0
          atomicOr(&g_dev_words[0], kStatusBadPaged);
          for (int x = 0; x < bytes; x += 16) st_shared16(dst + x, make_uint4(0u, 0u, 0u, 0u));
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        }
        __syncwarp();
      }
      if (lane == 0) {
        if (which == 0)
          words->step[c % kStepWords] = make_int4(g.walk.p0 - tok0, g.seq.hist - tok0, g.walk.rows,
                                                  (i == 0 ? 1 : 0) | (i == g.n - 1 ? 2 : 0));
        mbar_arrive_expect_tx(ring.full(st),
                              (uint32_t)((npg - __popc(bad & 0xffffu)) * ((T::CODEB + T::SCALEB) << ts)));
      }
      __syncwarp();
      if (mine && good) {
        const uint8_t* tile = pool.pages + page * pool.page_stride +
                              ((long long)g.h * pool.tiles + ((tok0 & (ps - 1)) >> ts)) * pool.tile_bytes;
        bulk_load(dst, tile + (part ? T::scales(ts, which, 0) : T::codes(ts, which, 0)), (uint32_t)bytes,
                  ring.full(st));
      }
      ++c;
      if (++st == ring.stages()) {
        st = 0;
        ++round;
      }
    }
  }
  // every copy lands before the CTA ends
  if (lane == 0) drain_copies(ring.full(0), ring.stages(), c);
  __syncwarp();
}

// The keys' (which = 0, with each item's Q tile) or the values' tiles from the
// codes, by kUnpackWarps warps, this one the `part`-th.  A lane takes 32
// channels of a key at a time, 16 bytes of codes and two scales, and stores them
// as bf16 where the bulk-tensor copy of a bf16 pool would put them: 8 lanes'
// 16-byte stores meet all banks.  Rows behind the last key hold what some codes
// stand for, finite numbers that P's zeros meet.
template <int D>
__device__ void paged_unpack(const CUtensorMap* tm_q, uint32_t steps, const PagedWords* words, uint32_t base,
                             const WaitCtx& wt, int which, int part) {
  using C = Cfg<D>;
  using U = PagedCfg<D, true>;
  using T = Q4Tile<D>;
  constexpr int LANES = D < 64 ? 1 : 2;   // that share a row of a chunk of channels
  constexpr int ROWS = 32 / LANES;        // a warp's rows of a load
  constexpr int STEP = ROWS * kUnpackWarps;
  // Loads a round of the loop.  At d = 128 the unpacking itself bounds the
  // kernel, and four in flight at once are faster (chunks of 100 to 700 tokens
  // 111 us, 122 with two, 127 with one); else what counts is that the kernel's
  // loops together fit the instruction cache (candidates 364 us with four, 339
  // with two, 338 with one).
  constexpr int GROUPS = D == 128 ? 4 : 2;
  constexpr int ROUNDS = kBN / STEP / GROUPS;
  const RawRing<D> ring{base, which};
  const uint32_t bars = base + C::BAR_OFF;
  auto bar = [&](int i) { return bars + 8u * (uint32_t)i; };
  const int lane = threadIdx.x & 31;
  const int row0 = part * ROWS + lane / LANES;  // and every STEP rows after it
  const int sub = lane % LANES;                 // which 32 channels of the chunk
  // the rows' swizzle is the same for all of a lane's rows
  const int turn = C::ROWB == 128 ? (row0 & 7) : ((row0 >> 1) & 3);
  const uint32_t dst = base + (which ? C::V_OFF : C::K_OFF) + row0 * C::ROWB + (((4 * sub) ^ turn) << 4);
  const uint32_t src = row0 * T::CODEB + 16 * sub;
  const uint32_t src_sc = kBN * T::CODEB + row0 * T::SCALEB + 2 * sub;
  const int slots = which ? C::P : U::KP;
  uint32_t qc = 0, round = 0, raw_round = 0;
  int slot = 0, raw = 0, j = 0;  // the tile's slot, the codes' stage, c mod P
  for (uint32_t c = 0; c < steps; ++c) {
    bool ok = wait_one(ring.full(raw), raw_round & 1u, wt, which ? kSiteVFull : kSiteKFull);
    if (lane == 0 && ok) {
      if (which == 0) {
        if (part == 0 && read_step(words, c).first()) {
          const int qs = (int)(qc % C::QS);
          ok = wait_one(bar(C::B_QEMPTY + qs), ((qc / C::QS) & 1u) ^ 1u, wt, kSiteQEmpty);
          if (ok) {
            const volatile PagedItem& x = words->item[qc % kItemWords];
            const int h = x.h, row = x.row0;
            mbar_arrive_expect_tx(bar(C::B_QFULL + qs), C::TILEB);
#pragma unroll
            for (int ch = 0; ch < C::NCHUNK; ++ch)
              tma_load_3d(base + C::Q_OFF + qs * C::TILEB + ch * C::CHUNKB, tm_q, bar(C::B_QFULL + qs),
                          ch * C::CHUNK, h, row);
            ++qc;
          }
        }
        // QK(c - KP) done: its S buffer is written
        if (ok && round > 0)
          ok = wait_one(bar(C::B_SFULL + (int)((c - U::KP) % C::P)), ((c - U::KP) / C::P) & 1u, wt, kSiteKEmpty);
      } else {
        ok = wait_one(bar(C::B_QKREADY + j), (c / C::P) & 1u, wt, kSiteVEmpty);
      }
    }
    if (!__all_sync(0xffffffffu, ok)) break;
#pragma unroll 1
    for (int q = 0; q < C::NCHUNK * ROUNDS; ++q) {
      const int ch = q / ROUNDS, first = (q % ROUNDS) * GROUPS * STEP;
      const uint32_t from = ring.stage(raw) + src + first * T::CODEB + 32 * ch;
      const uint32_t from_sc = ring.stage(raw) + src_sc + first * T::SCALEB + 4 * ch;
      const uint32_t to = dst + slot * C::TILEB + first * C::ROWB + ch * C::CHUNKB;
      uint4 u[GROUPS];
      uint32_t sc[GROUPS];
#pragma unroll
      for (int x = 0; x < GROUPS; ++x) {
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(u[x].x), "=r"(u[x].y), "=r"(u[x].z), "=r"(u[x].w)
                     : "r"(from + x * STEP * T::CODEB)
                     : "memory");
        asm volatile("ld.shared.u16 %0, [%1];" : "=r"(sc[x]) : "r"(from_sc + x * STEP * T::SCALEB) : "memory");
      }
      if (D == 128 && q == C::NCHUNK * ROUNDS - 1) {
        // the stage is read: its next codes may come while these are converted
        // (chunks of 100 to 700 tokens 110 us, 123 without; at d = 64, with four
        // stages, the candidates would take 431 us, 364 without)
        __syncwarp();
        if (lane == 0) mbar_arrive(ring.empty(raw));
      }
#pragma unroll
      for (int x = 0; x < GROUPS; ++x) {
        const Q4Scale s0 = q4_scale(sc[x] & 255u), s1 = q4_scale(sc[x] >> 8);
        const uint32_t st = to + x * STEP * C::ROWB;
        st_shared16(st, q4_word(u[x].x, s0));
        st_shared16(st ^ 16u, q4_word(u[x].y, s0));
        st_shared16(st ^ 32u, q4_word(u[x].z, s1));
        st_shared16(st ^ 48u, q4_word(u[x].w, s1));
      }
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
    if (lane == 0) {
      if (D != 128) mbar_arrive(ring.empty(raw));
      mbar_arrive(bar((which ? C::B_VFULL : C::B_QKREADY) + j));
    }
    if (++j == C::P) j = 0;
    if (++slot == slots) {
      slot = 0;
      ++round;
    }
    if (++raw == ring.stages()) {
      raw = 0;
      ++raw_round;
    }
  }
  // every copy lands before the CTA ends
  if (which == 0 && lane == 0) drain_copies(bar(C::B_QFULL), C::QS, qc);
  __syncwarp();
}

// QK issuer: as role_mma_qk.
template <int D, bool Q4>
__device__ void paged_mma_qk(const PagedFwdArgs& a, uint32_t steps, const PagedWords* words,
                             uint32_t base, uint32_t tmem, const WaitCtx& wt) {
  using C = Cfg<D>;
  constexpr int P = C::P;
  const uint32_t bars = base + C::BAR_OFF;
  auto bar = [&](int i) { return bars + 8u * (uint32_t)i; };
  constexpr uint32_t IDESC_QK = make_idesc(kBM, kBN, 0);
  constexpr int QK_STEPS = D / 16;
  constexpr int STEPS_PER_CHUNK = C::CHUNK / 16;
  const uint64_t q_desc0 = smem_desc(base + C::Q_OFF, 16, C::ATOMB, C::LAYOUT);
  const uint64_t k_desc0 = smem_desc(base + C::K_OFF, 16, C::ATOMB, C::LAYOUT);
  bool ok = true;
  if (a.debug_flags & kDebugUnsignalledWait) ok = wait_one(bar(C::B_DRAIN), 0u, wt, kSiteUnsignalled);
  if (!ok) steps = 0;
  uint32_t tc = 0, it = 0;
  uint32_t ph = 0;
  constexpr int KP = PagedCfg<D, Q4>::KP;
  for (int J = 0; tc < steps; J = J + 1 == P ? 0 : J + 1) {
    const int kslot = KP == P ? J : (int)(tc % KP);
    const int qs = C::QS == 1 ? 0 : (int)(it & 1u);
    if (!(ok = wait_one(bar(C::B_QKREADY + J), ph, wt, kSiteKFull))) break;
    const PagedStep st = read_step(words, tc);
    if (st.first() && !(ok = wait_one(bar(C::B_QFULL + qs), (it / C::QS) & 1u, wt, kSiteQFull))) break;
    tc_fence_after();
    const int cols = st.cols();
    const uint32_t s_tmem = pin32(tmem + (uint32_t)(J * 128));
    const uint32_t idesc = pin32(cols == kBN ? IDESC_QK : make_idesc(kBM, cols, 0));
    const uint64_t qd0 = q_desc0 + (uint64_t)((qs * C::TILEB) >> 4);
    uint64_t qd[QK_STEPS], kd[QK_STEPS];
#pragma unroll
    for (int kk = 0; kk < QK_STEPS; ++kk) {
      const uint32_t off = (kk / STEPS_PER_CHUNK) * C::CHUNKB + (kk % STEPS_PER_CHUNK) * 32;
      qd[kk] = pin64(qd0 + (uint64_t)(off >> 4));
      kd[kk] = pin64(k_desc0 + (uint64_t)((kslot * C::TILEB + off) >> 4));
    }
    mma_ss_c<0>(s_tmem, qd[0], kd[0], idesc);
#pragma unroll
    for (int kk = 1; kk < QK_STEPS; ++kk) mma_ss_c<1>(s_tmem, qd[kk], kd[kk], idesc);
    mma_commit(bar(C::B_SFULL + J));
    if (st.last()) {
      mma_commit(bar(C::B_QEMPTY + qs));
      ++it;
    }
    ++tc;
    if (J == P - 1) ph ^= 1u;
  }
  // every product is done before TMEM is freed, also where the SiLU warps have
  // given up
  mma_commit(bar(C::B_DRAIN));
  wait_drain(bar(C::B_DRAIN), 0);
}

// PV issuer: as role_mma_pv, with the block that holds the tile's last keys
// cut at the first key that no row sees.
// Q4: the values come from codes.  Rows behind the last key hold what some
// bytes stand for, but whatever bytes do is finite, and P is zero there: they
// add nothing and need no clearing.
template <int D, bool Q4>
__device__ void paged_mma_pv(uint32_t steps, const PagedWords* words, uint32_t base, uint32_t tmem,
                             const WaitCtx& wt) {
  using C = Cfg<D>;
  constexpr int P = C::P;
  const uint32_t bars = base + C::BAR_OFF;
  auto bar = [&](int i) { return bars + 8u * (uint32_t)i; };
  constexpr uint32_t IDESC_PV = make_idesc(kBM, D, 1);
  const uint64_t v_desc0 = smem_desc(base + C::V_OFF, C::CHUNKB, C::ATOMB, C::LAYOUT);
  bool ok = true;
  uint32_t tc = 0, it = 0;
  uint32_t ph = 0;

  auto issue_pv = [&](int J, auto hc, int ob, int cols, bool start) {
    constexpr int H = decltype(hc)::value;
    const uint32_t o_tmem = pin32(tmem + C::O_COL + (uint32_t)(ob * D));
    uint32_t pa[8];
    uint64_t vb[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int kk = 4 * H + i;
      pa[2 * i] = pin32(tmem + (uint32_t)(J * 128 + 16 * kk));  // P_hi, then P_lo
      pa[2 * i + 1] = pin32(tmem + (uint32_t)(J * 128 + 16 * kk + 8));
      vb[i] = pin64(v_desc0 + (uint64_t)((J * C::TILEB + kk * 2 * C::ATOMB) >> 4));
    }
    if (cols == kBN && (H == 1 || !start)) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        mma_ts_c<1>(o_tmem, pa[2 * i], vb[i], IDESC_PV);
        mma_ts_c<1>(o_tmem, pa[2 * i + 1], vb[i], IDESC_PV);
      }
    } else {
      const int n_steps = (cols - 64 * H) / 16;
      const bool first = H == 0 && start;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (i < n_steps) {
          if (i == 0 && first)
            mma_ts_c<0>(o_tmem, pa[0], vb[0], IDESC_PV);
          else
            mma_ts_c<1>(o_tmem, pa[2 * i], vb[i], IDESC_PV);
          mma_ts_c<1>(o_tmem, pa[2 * i + 1], vb[i], IDESC_PV);
        }
      }
    }
  };

  bool pa_ready = false, v_ready = false;
  for (int J = 0; tc < steps; J = J + 1 == P ? 0 : J + 1) {
    const int JN = J + 1 == P ? 0 : J + 1;
    const int ob = C::OB == 1 ? 0 : (int)(it & 1u);
    if (!pa_ready && !(ok = wait_one(bar(C::B_PFULL + J), ph, wt, kSitePFull))) break;
    const PagedStep st = read_step(words, tc);
    const int cols = st.cols();
    if (st.first() &&
        !(ok = wait_one(bar(C::B_OEMPTY + ob), ((it / C::OB) & 1u) ^ 1u, wt, kSiteOEmpty)))
      break;
    if (!v_ready && !(ok = wait_one(bar(C::B_VFULL + J), ph, wt, kSiteVFull))) break;
    if (!Q4 && st.end() < cols) {
      // keys that no row sees: their P is zero, their V may be anything
      const uint32_t v_addr = base + C::V_OFF + J * C::TILEB;
#pragma unroll
      for (int ch = 0; ch < C::NCHUNK; ++ch) {
        const uint32_t z0 = v_addr + ch * C::CHUNKB + st.end() * C::ROWB;
        const uint32_t z1 = v_addr + ch * C::CHUNKB + cols * C::ROWB;
        for (uint32_t z = z0; z < z1; z += 16)
          asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(z), "r"(0) : "memory");
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    tc_fence_after();
    const uint32_t npar = J + 1 == P ? ph ^ 1u : ph;
    pa_ready = mbar_test(bar(C::B_PFULL + JN), npar);
    v_ready = mbar_test(bar(C::B_VFULL + JN), npar);
    issue_pv(J, std::integral_constant<int, 0>{}, ob, cols, st.first());
    issue_pv(J, std::integral_constant<int, 1>{}, ob, cols, st.first());
    mma_commit(bar(C::B_QKREADY + J));
    if (st.last()) {
      mma_commit(bar(C::B_OFULL + ob));
      ++it;
    }
    ++tc;
    if (J == P - 1) ph ^= 1u;
  }
  mma_commit(bar(C::B_DRAIN + 1));
  wait_drain(bar(C::B_DRAIN + 1), 0);
  if (!Q4 && !ok) arrive_for_dropped_pv<P>(bar(C::B_QKREADY), tc);
}

// SiLU warpgroups: as role_silu's wide form.  A masked block keeps key k for
// the row at lim iff k <= lim and (k < lim_hist or k == lim); 16-key steps
// none of whose keys a warp's rows keep are zeros without a load.
template <int D>
__device__ void paged_silu(const PagedFwdArgs& a, uint32_t steps, const PagedWords* words, uint32_t base,
                           uint32_t tmem, const WaitCtx& wt, int warp, int lane) {
  using C = Cfg<D>;
  constexpr int P = C::P;
  const uint32_t bars = base + C::BAR_OFF;
  auto bar = [&](int i) { return bars + 8u * (uint32_t)i; };
  const int wg = (warp - kEwWarp0) >> 2;
  const int e = wg >> 1, half = wg & 1;  // every other step, half of its keys
  const int quarter = warp & 3;
  const uint32_t lane_base = tmem + ((uint32_t)(quarter * 32) << 16);
  const float2 ha2 = make_float2(a.half_alpha, a.half_alpha);
  for (uint32_t tc = (uint32_t)e; tc < steps; tc += 2) {
    const int j = (int)(tc % P);
    {
      const bool ok = wait_one(bar(C::B_SFULL + j), (tc / P) & 1u, wt, kSiteSFull);
      if (!__all_sync(0xffffffffu, ok)) return;
    }
    tc_fence_after();
    const PagedStep st = read_step(words, tc);
    const uint32_t t_s = lane_base + (uint32_t)(j * 128);
    if (quarter * 32 < st.rows) {
      if (st.plain()) {
        uint32_t w0[16], w1[16];
        const uint32_t t_h = t_s + 64u * (uint32_t)half;
        tmem_ld16_async(t_h, w0);
        tmem_wait_ld16(w0);
#pragma unroll 1
        for (int u = 0; u < 4; u += 2) {
          tmem_ld16_async(t_h + 16u * (u + 1), w1);
          silu_store16<0>(w0, ha2, 0, 0, t_h + 16u * u);
          tmem_wait_ld16(w1);
          if (u + 2 < 4) tmem_ld16_async(t_h + 16u * (u + 2), w0);
          silu_store16<0>(w1, ha2, 0, 0, t_h + 16u * (u + 1));
          if (u + 2 < 4) tmem_wait_ld16(w0);
        }
      } else {
        const int cols = st.cols();
        // the warp's rows stand at lim0 .. lim0 + 31, this lane's at lim0 + lane
        const int lim0 = st.lim + 32 * quarter;
        const int hist0 = st.hist;
#pragma unroll 1
        for (int k = 64 * half; k < 64 * half + 64 && k < cols; k += 16) {
          const uint32_t t_k = t_s + (uint32_t)k;
          uint32_t s[16];
          if (k > lim0 + 31 || (k >= hist0 && k + 16 <= lim0)) {
#pragma unroll
            for (int m = 0; m < 16; ++m) s[m] = 0u;
            tmem_st16(t_k, s);
          } else {
            tmem_ld16_async(t_k, s);
            tmem_wait_ld16(s);
            silu_store16<2>(s, ha2, lim0 + lane - k, hist0 - k, t_k);
          }
        }
      }
      tmem_wait_st();
    }
    tc_fence_before();
    mbar_arrive(bar(C::B_PFULL + j));
  }
}

// Epilogue: O x inv_n -> bf16 rows, or this CTA's part of a cut item, fp32 as
// [D / 4][128 rows] float4 (consecutive lanes, consecutive 16 bytes), with a
// note of the item for paged_join.
template <int D>
__device__ void paged_epilogue(const PagedFwdArgs& a, uint32_t steps, PagedWords* words, uint32_t base,
                               uint32_t tmem, const WaitCtx& wt, int warp, int lane) {
  using C = Cfg<D>;
  const uint32_t bars = base + C::BAR_OFF;
  auto bar = [&](int i) { return bars + 8u * (uint32_t)i; };
  const int quarter = warp & 3;
  const int row = quarter * 32 + lane;
  const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
  for (uint32_t it = 0, done = 0; done < steps; ++it) {
    const int ob = (int)(it % C::OB);
    if (!wait_warp(bar(C::B_OFULL + ob), (it / C::OB) & 1u, wt, kSiteOFull)) return;
    tc_fence_after();
    const volatile PagedItem& x = words->item[it % kItemWords];
    const PagedItem g{x.row0, x.h, x.rows, x.blocks, x.c0, x.parts};
    done += (uint32_t)g.blocks;
    const uint32_t o_t = tmem + lane_off + C::O_COL + (uint32_t)(ob * D);
    const bool live = row < g.rows;
    if (g.parts == 1) {
      uint4* dst = reinterpret_cast<uint4*>(
          a.out + ((size_t)(g.row0 + row) * (size_t)a.w.heads + (size_t)g.h) * D);
      // 64 columns at a time (the registers of 768 threads); the O buffer is
      // released before the last ones are stored
      constexpr int PIECE = D < 64 ? D : 64;
#pragma unroll
      for (int c0 = 0; c0 < D; c0 += PIECE) {
        uint32_t packed[PIECE / 2];
#pragma unroll
        for (int cc = 0; cc < PIECE / 32; ++cc) {
          uint32_t o[32];
          tmem_ld32(o_t + (uint32_t)c0 + 32u * cc, o);
#pragma unroll
          for (int m = 0; m < 16; ++m)
            packed[16 * cc + m] =
                pack_bf16x2(__uint_as_float(o[2 * m]) * a.inv_n, __uint_as_float(o[2 * m + 1]) * a.inv_n);
        }
        if (c0 + PIECE == D) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(C::B_OEMPTY + ob));
        }
        if (live) {
#pragma unroll
          for (int u = 0; u < PIECE / 8; ++u)
            dst[c0 / 8 + u] =
                make_uint4(packed[4 * u], packed[4 * u + 1], packed[4 * u + 2], packed[4 * u + 3]);
        }
      }
      continue;
    }
    const int starts = g.c0 == (int)blockIdx.x ? 1 : 0;
    float4* mine = paged_part<D>(a, blockIdx.x, starts) + row;
#pragma unroll 1
    for (int cc = 0; cc < D / 32; ++cc) {
      uint32_t o[32];
      tmem_ld32(o_t + 32u * cc, o);
      if (live) {
#pragma unroll
        for (int m = 0; m < 8; ++m)
          __stcg(mine + (8 * cc + m) * kBM,
                 make_float4(__uint_as_float(o[4 * m]), __uint_as_float(o[4 * m + 1]),
                             __uint_as_float(o[4 * m + 2]), __uint_as_float(o[4 * m + 3])));
      }
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(C::B_OEMPTY + ob));
    if (row == 0) words->cut[starts] = g;
  }
}

// Once all roles are done: the last CTA to arrive at a cut item (the one that
// an earlier CTA starts, the one that this CTA starts) sums its parts in the
// CTAs' order, with all its threads, so that the result does not depend on
// who is last.  One fence a CTA, after the barrier and so for all the warps'
// stores.
template <int D>
__device__ void paged_join(const PagedFwdArgs& a, PagedWords* words, bool dead) {
  if (words->cut[0].parts == 0 && words->cut[1].parts == 0) return;
  if (threadIdx.x == 0) {
    __threadfence();
    unsigned last = 0;
    for (int k = 0; k < 2; ++k) {
      const PagedItem& g = words->cut[k];
      if (!g.parts || dead || atomicAdd(a.counters + g.c0, 1u) != (unsigned)(g.parts - 1)) continue;
      last |= 1u << k;
      a.counters[g.c0] = 0;  // ready for the next launch
    }
    words->last = last;
  }
  __syncthreads();
  const unsigned last = words->last;
  if (last) __threadfence();
#pragma unroll 1
  for (int k = 0; k < 2; ++k) {
    if (!(last >> k & 1u)) continue;
    const PagedItem g = words->cut[k];
    for (int x = threadIdx.x; x < g.rows * (D / 4); x += blockDim.x) {
      const int c4 = x / g.rows, row = x - c4 * g.rows;
      const int at = c4 * kBM + row;
      float4 v = __ldcg(paged_part<D>(a, g.c0, 1) + at);
#pragma unroll 1
      for (int i = 1; i < g.parts; i += 8) {  // eight loads in flight
        float4 y[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
          y[j] = i + j < g.parts ? __ldcg(paged_part<D>(a, g.c0 + i + j, 0) + at)
                                 : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          v.x += y[j].x;
          v.y += y[j].y;
          v.z += y[j].z;
          v.w += y[j].w;
        }
      }
      *reinterpret_cast<uint2*>(a.out + ((size_t)(g.row0 + row) * (size_t)a.w.heads + (size_t)g.h) * D +
                                4 * c4) =
          make_uint2(pack_bf16x2(v.x * a.inv_n, v.y * a.inv_n), pack_bf16x2(v.z * a.inv_n, v.w * a.inv_n));
    }
  }
}

template <int D, class SRC>
__global__ void __launch_bounds__(kPagedThreadsOf<SRC>, 1)
    hstu_fwd_paged_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ SRC src,
                          const PagedFwdArgs a) {
  using C = Cfg<D>;
  constexpr bool Q4 = kHeldInQ4<SRC>;
  constexpr int WARPS = kPagedThreadsOf<SRC> / 32;
  extern __shared__ uint8_t smem_raw[];
  __shared__ PagedStart<WARPS> start;
  __shared__ PagedWords words;
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base - raw);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::MISC_OFF);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::MISC_OFF + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t bars = base + C::BAR_OFF;
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::NBARS; ++i) mbar_init(bars + 8u * i, paged_arrivals<D, Q4>(i));
    for (int j = 0; j < C::P; ++j) mbar_arrive(bars + 8u * (C::B_QKREADY + j));
    if constexpr (Q4) {
      for (int which = 0; which < 2; ++which) {
        const RawRing<D> ring{base, which};
        for (int s = 0; s < ring.stages(); ++s) {
          mbar_init(ring.full(s), 1);
          mbar_init(ring.empty(s), kUnpackWarps);
        }
      }
    }
    *abort_flag = 0;
    words.cut[0].parts = words.cut[1].parts = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  after_previous_kernel();
  PagedWork w = a.w;
  PagedCursor from;
  PagedSeg first;
  int n_steps;
  // a CTA without work leaves before it allocates TMEM
  if (!paged_locate<WARPS, true>(a.p, &w, &start, &g_dev_words[0], &from, &first, &n_steps)) return;
  if (warp == kMmaWarpQK) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(tmem_slot)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const WaitCtx wt{a.timeout_ns, abort_flag};
  const uint32_t steps = (uint32_t)n_steps;
  if (warp == kTmaWarpK || warp == kTmaWarpV) {
    if constexpr (Q4)
      paged_copy_codes<D>(src, a, w, from, first, &words, base, wt, warp == kTmaWarpV);
    else if (warp == kTmaWarpK)
      paged_producer<D, true>(&src.k, &tm_q, a, w, from, first, &words, base, wt);
    else
      paged_producer<D, false>(&src.v, &tm_q, a, w, from, first, &words, base, wt);
  } else if (Q4 && warp < 2 * kUnpackWarps) {
    if constexpr (Q4) paged_unpack<D>(&tm_q, steps, &words, base, wt, warp & 1, warp >> 1);
  } else if (warp == kMmaWarpQK) {
    if (lane == 0) paged_mma_qk<D, Q4>(a, steps, &words, base, tmem, wt);
    __syncwarp();
  } else if (warp == kMmaWarpPV) {
    if (lane == 0) paged_mma_pv<D, Q4>(steps, &words, base, tmem, wt);
    __syncwarp();
  } else if (warp >= kEwWarp0 && warp < kEwWarp0 + kSiluWarps) {
    paged_silu<D>(a, steps, &words, base, tmem, wt, warp, lane);
  } else {
    paged_epilogue<D>(a, steps, &words, base, tmem, wt, warp, lane);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarpQK) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "r"(kTmemCols)
                 : "memory");
  }
  paged_join<D>(a, &words, *abort_flag != 0);
}

template <int D, class SRC>
cudaError_t launch_paged_d(const CUtensorMap& tq, const SRC& src, const PagedFwdArgs& a, int grid,
                           cudaStream_t stream) {
  constexpr int SMEM = PagedCfg<D, kHeldInQ4<SRC>>::SMEM;
  static DeviceOnce once;
  const cudaError_t e = once.run([] {
    return cudaFuncSetAttribute(hstu_fwd_paged_kernel<D, SRC>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                SMEM);
  });
  if (e != cudaSuccess) return e;
  return launch_after(hstu_fwd_paged_kernel<D, SRC>, grid, kPagedThreadsOf<SRC>, SMEM, stream, tq,
                      src, a);
}
template <class SRC>
cudaError_t launch_paged(int d, const CUtensorMap& tq, const SRC& src, const PagedFwdArgs& a, int grid,
                         cudaStream_t stream) {
  switch (d) {
    case 32: return launch_paged_d<32>(tq, src, a, grid, stream);
    case 64: return launch_paged_d<64>(tq, src, a, grid, stream);
    case 128: return launch_paged_d<128>(tq, src, a, grid, stream);
    default: return cudaErrorInvalidValue;
  }
}
