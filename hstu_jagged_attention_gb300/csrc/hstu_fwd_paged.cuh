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
// ahead of the epilogue: 16 item words are enough.
constexpr int kStepWords = 8, kItemWords = 16;
constexpr int kPagedThreads = 768;  // four SiLU warpgroups, the wide P layout, at every d
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

// QK issuer: as role_mma_qk.
template <int D>
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
  for (int J = 0; tc < steps; J = J + 1 == P ? 0 : J + 1) {
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
      kd[kk] = pin64(k_desc0 + (uint64_t)((J * C::TILEB + off) >> 4));
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
template <int D>
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
    if (st.end() < cols) {
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
  if (!ok) arrive_for_dropped_pv<P>(bar(C::B_QKREADY), tc);
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
    if (threadIdx.x == 0) words->cut[starts] = g;
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

template <int D>
__global__ void __launch_bounds__(kPagedThreads, 1)
    hstu_fwd_paged_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                          const __grid_constant__ CUtensorMap tm_v, const PagedFwdArgs a) {
  using C = Cfg<D>;
  constexpr int WARPS = kPagedThreads / 32;
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
    for (int i = 0; i < C::NBARS; ++i) mbar_init(bars + 8u * i, C::arrivals(i, true));
    for (int j = 0; j < C::P; ++j) mbar_arrive(bars + 8u * (C::B_QKREADY + j));
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
  if (warp == kTmaWarpK) {
    paged_producer<D, true>(&tm_k, &tm_q, a, w, from, first, &words, base, wt);
  } else if (warp == kTmaWarpV) {
    paged_producer<D, false>(&tm_v, &tm_q, a, w, from, first, &words, base, wt);
  } else if (warp == kMmaWarpQK) {
    if (lane == 0) paged_mma_qk<D>(a, steps, &words, base, tmem, wt);
    __syncwarp();
  } else if (warp == kMmaWarpPV) {
    if (lane == 0) paged_mma_pv<D>(steps, &words, base, tmem, wt);
    __syncwarp();
  } else if (warp >= kEwWarp0) {
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

template <int D>
cudaError_t launch_paged_d(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                           const PagedFwdArgs& a, int grid, cudaStream_t stream) {
  using C = Cfg<D>;
  static DeviceOnce once;
  const cudaError_t e = once.run([] {
    return cudaFuncSetAttribute(hstu_fwd_paged_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                C::SMEM_LAUNCH);
  });
  if (e != cudaSuccess) return e;
  return launch_after(hstu_fwd_paged_kernel<D>, grid, kPagedThreads, C::SMEM_LAUNCH, stream, tq, tk,
                      tv, a);
}
