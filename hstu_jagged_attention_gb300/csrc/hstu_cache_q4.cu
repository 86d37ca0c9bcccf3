// The paged K/V cache held in 4 bits: appending keys and values to it (rotated,
// then quantised), reading them back, and the attention of new tokens over it.
//
//   append   page_table and rotation as the bf16 cache's (hstu_cache.cu);
//            what is held of a bf16 number is hstu_q4.cuh's
//   attention
//            out[t,h,:] = inv_n sum_j silu(alpha q[t,h,:].K_j) V_j over the
//            keys and values held
//
// (ai6s.net post section 1 for the formula; HSTU paper section 3.4: the
// history's keys and values are cached and serve every microbatch.)
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "hstu_attn.h"
#include "hstu_internal.h"
#include "hstu_paged.cuh"
#include "hstu_ptx.cuh"
#include "hstu_q4.cuh"
#include "hstu_step.cuh"

namespace hstu {
namespace {

constexpr int kQ4Threads = 256;

// Where a thread of the append and of the reading works: a group of 16
// channels of one head of one token.  A warp takes consecutive tokens of one
// head, whose codes are consecutive bytes.
struct Q4Unit {
  long long t;
  int h, g;
};
template <int D>
__device__ __forceinline__ Q4Unit q4_unit(unsigned block, int heads) {
  constexpr int G = D / kQ4Group, TOKENS = 32 / G;
  const long long w = ((long long)block * kQ4Threads + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  const long long tb = w / heads;
  return Q4Unit{tb * TOKENS + lane / G, (int)(w - tb * heads), lane % G};
}
template <int D>
long long q4_blocks(long long rows, int heads) {
  constexpr int TOKENS = 32 / (D / kQ4Group);
  return ((rows + TOKENS - 1) / TOKENS * heads * 32 + kQ4Threads - 1) / kQ4Threads;
}

// The first CTAs check a sequence a thread: one that contradicts itself may
// have no row.
__device__ __forceinline__ bool q4_checks(const PagedView& p, unsigned check_ctas, unsigned* status) {
  if (blockIdx.x >= check_ctas) return false;
  const long long b = (long long)blockIdx.x * kQ4Threads + threadIdx.x;
  PagedSeq s;
  if (b < p.batch && !paged_seq(p, (int)b, &s)) atomicOr(status, kStatusBadPaged);
  return true;
}

// Byte of tile row 0 of token slot `slot`, and its row there.
__device__ __forceinline__ long long q4_tile(const Q4Pool& pool, int page_shift, long long slot, int h, int* r) {
  const int in_page = (int)(slot & ((1 << page_shift) - 1));
  *r = in_page & ((1 << pool.tile_shift) - 1);
  return (slot >> page_shift) * pool.page_stride +
         ((long long)h * pool.tiles + (in_page >> pool.tile_shift)) * pool.tile_bytes;
}

// 8 channels c .. c + 7 of a head, x, rotated with its partner block y where
// the channels turn in halves.  The products are rounded one by one, as a
// plain form does: what is quantised then is the same number, not one beside
// it across a border.
__device__ __forceinline__ uint4 q4_turn(const uint4& x, const uint4& y, const float* tab, int c, int rot,
                                         bool pairs) {
  F8 a = unpack8(x);
  const int half = rot >> 1;
  if (pairs) {
    const float4 cs = __ldg(reinterpret_cast<const float4*>(tab + (c >> 1)));
    const float4 sn = __ldg(reinterpret_cast<const float4*>(tab + half + (c >> 1)));
    const float cc[4] = {cs.x, cs.y, cs.z, cs.w}, ss[4] = {sn.x, sn.y, sn.z, sn.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float u = a.f[2 * i], v = a.f[2 * i + 1];
      a.f[2 * i] = __fsub_rn(__fmul_rn(u, cc[i]), __fmul_rn(v, ss[i]));
      a.f[2 * i + 1] = __fadd_rn(__fmul_rn(v, cc[i]), __fmul_rn(u, ss[i]));
    }
  } else {
    const bool first = c < half;
    const float* at = tab + (first ? c : c - half);
    const F8 b = unpack8(y);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float4 cs = __ldg(reinterpret_cast<const float4*>(at) + k);
      const float4 sn = __ldg(reinterpret_cast<const float4*>(at + half) + k);
      const float cc[4] = {cs.x, cs.y, cs.z, cs.w}, ss[4] = {sn.x, sn.y, sn.z, sn.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float s = first ? -ss[i] : ss[i];
        a.f[4 * k + i] = __fadd_rn(__fmul_rn(a.f[4 * k + i], cc[i]), __fmul_rn(b.f[4 * k + i], s));
      }
    }
  }
  return pack8(a);
}

__device__ __forceinline__ uint4 load16(const uint16_t* p) { return *reinterpret_cast<const uint4*>(p); }

template <int D>
__global__ void __launch_bounds__(kQ4Threads) append_q4_kernel(const AppendArgs a, const Q4Pool pool) {
  using T = Q4Tile<D>;
  after_previous_kernel();
  if (q4_checks(a.p, a.check_ctas, a.status)) return;
  const Q4Unit u = q4_unit<D>(blockIdx.x - a.check_ctas, a.heads);
  if (u.t >= a.p.rows) return;
  const int t = (int)u.t, c0 = kQ4Group * u.g, c1 = c0 + 8;
  const bool turn = a.table && c0 < a.rot;
  const int half = a.rot >> 1;
  const bool halves = turn && !a.pairs;
  // the partners' blocks, where channels turn in halves
  const int y0 = !halves ? c0 : c0 < half ? c0 + half : c0 - half;
  const int y1 = !halves ? c1 : c1 < half ? c1 + half : c1 - half;
  const long long at = (long long)u.h * D;
  const uint16_t* kr = a.k + t * a.k_stride + at;
  const uint16_t* vr = a.v + t * a.v_stride + at;
  const int total = a.p.q_offsets[a.p.batch];
  uint4 k0 = load16(kr + c0), k1 = load16(kr + c1), kp0{}, kp1{}, q0{}, q1{}, qp0{}, qp1{};
  const uint4 v0 = load16(vr + c0), v1 = load16(vr + c1);
  if (halves) {
    kp0 = load16(kr + y0);
    kp1 = load16(kr + y1);
  }
  if (a.q) {
    const uint16_t* qr = a.q + t * a.q_stride + at;
    q0 = load16(qr + c0);
    q1 = load16(qr + c1);
    if (halves) {
      qp0 = load16(qr + y0);
      qp1 = load16(qr + y1);
    }
  }
  if (t >= total) return;  // a row behind the last sequence
  PagedSeq s;
  const int b = paged_find(a.p, t);
  if (b < 0 || !paged_seq(a.p, b, &s)) return;  // before the first sequence, or of one that is reported
  const int pos = s.kv - s.qn + (t - s.q0);
  const long long slot = paged_slot(a.p, b, pos);
  const int turned_at = pos < s.hist ? pos : s.hist;  // a candidate stands right behind the history
  if (slot < 0 || (a.table && turned_at >= a.positions)) {
    atomicOr(a.status, kStatusBadPaged);
    return;
  }
  if (turn) {
    const float* tab = a.table + (long long)turned_at * a.rot;
    k0 = q4_turn(k0, kp0, tab, c0, a.rot, a.pairs);
    k1 = q4_turn(k1, kp1, tab, c1, a.rot, a.pairs);
    if (a.q) {
      q0 = q4_turn(q0, qp0, tab, c0, a.rot, a.pairs);
      q1 = q4_turn(q1, qp1, tab, c1, a.rot, a.pairs);
    }
  }
  int r;
  uint8_t* tile = pool.pages + q4_tile(pool, a.p.page_shift, slot, u.h, &r);
  uint32_t j;
  *reinterpret_cast<uint2*>(tile + T::codes(pool.tile_shift, 0, r) + 8 * u.g) = q4_quantise(k0, k1, &j);
  tile[T::scales(pool.tile_shift, 0, r) + u.g] = (uint8_t)j;
  *reinterpret_cast<uint2*>(tile + T::codes(pool.tile_shift, 1, r) + 8 * u.g) = q4_quantise(v0, v1, &j);
  tile[T::scales(pool.tile_shift, 1, r) + u.g] = (uint8_t)j;
  if (a.q) {
    uint4* qo = reinterpret_cast<uint4*>(a.q_out + (long long)t * a.heads * D + at + c0);
    qo[0] = q0;
    qo[1] = q1;
  }
}

template <int D>
__global__ void __launch_bounds__(kQ4Threads) read_q4_kernel(const ReadArgs a, const Q4Pool pool) {
  using T = Q4Tile<D>;
  after_previous_kernel();
  if (q4_checks(a.p, a.check_ctas, a.status)) return;
  const Q4Unit u = q4_unit<D>(blockIdx.x - a.check_ctas, a.heads);
  if (u.t >= a.p.rows) return;
  const int t = (int)u.t;
  PagedSeq s;
  const int b = paged_find(a.p, t);
  if (b < 0 || !paged_seq(a.p, b, &s)) return;
  const long long slot = paged_slot(a.p, b, s.kv - s.qn + (t - s.q0));
  uint2 kc{}, vc{};
  uint32_t kj = 0, vj = 0;
  if (slot < 0) {
    atomicOr(a.status, kStatusBadPaged);  // read as zeros
  } else {
    int r;
    const uint8_t* tile = pool.pages + q4_tile(pool, a.p.page_shift, slot, u.h, &r);
    kc = *reinterpret_cast<const uint2*>(tile + T::codes(pool.tile_shift, 0, r) + 8 * u.g);
    vc = *reinterpret_cast<const uint2*>(tile + T::codes(pool.tile_shift, 1, r) + 8 * u.g);
    kj = tile[T::scales(pool.tile_shift, 0, r) + u.g];
    vj = tile[T::scales(pool.tile_shift, 1, r) + u.g];
  }
  const Q4Scale ks = q4_scale(kj, kj), vs = q4_scale(vj, vj);
  const long long at = (long long)u.h * D + kQ4Group * u.g;
  uint4* ko = reinterpret_cast<uint4*>(a.k + t * a.k_stride + at);
  uint4* vo = reinterpret_cast<uint4*>(a.v + t * a.v_stride + at);
  ko[0] = q4_word(kc.x, ks);
  ko[1] = q4_word(kc.y, ks);
  vo[0] = q4_word(vc.x, vs);
  vo[1] = q4_word(vc.y, vs);
}

// ------------------------------------------------ attention of a few tokens
// As the bf16 cache's kernel of 16-row tiles (hstu_cache.cu): the last warp
// copies blocks of 128 keys with their values into a ring of shared-memory
// stages, one bulk copy a page, and the others take a part of the keys each.
// The codes become the products' B operands in registers:
//   S = Q K^T: a lane's operand of key n is channels 2 t .. and 2 t + 8 .. of
//     every 16; a sum over channels may take them in any order, so lane t has
//     the D / 4 consecutive channels whose codes it loads with one access, and
//     Q's operand the same ones;
//   O += P V: lane n's operand is channel n of keys 2 t, 2 t + 1, 2 t + 8 and
//     2 t + 9.  It loads D / 8 consecutive channels of its four keys, and one
//     byte permutation of two keys' words puts the keys side by side.  Which
//     channel a column of O is, and which key a column of S, is free, as long
//     as P's columns are V's rows: key 8 a + 4 e + (t + 2 e) % 4 for column
//     2 t + e of S's 8-key tile a lets neither load meet a bank twice (at d =
//     128, (t + e) % 4: K's do not, V's meet two).
// p is split into two bf16 terms; with up to 8 rows in a tile both terms are
// one operand, the second in its rows 8 .. 15.
// Keys past a row's last are masked by a select on p; whatever bytes lie
// there, as codes they are finite, and so add nothing.
template <int D>
struct Q4Cfg {
  static constexpr int WARPS = 8;
  static constexpr int THREADS = 32 * (WARPS + 1);
  static constexpr int KEYS = kStepKeys;
  static constexpr int KW = KEYS / WARPS;
  static constexpr int STAGEB = KEYS * q4_token_bytes(D);
  static constexpr int PER_SM = D == 128 ? 1 : 2;
  static constexpr int RING = 128 * 1024 / PER_SM;
  static constexpr int STAGES = RING / STAGEB < 15 ? RING / STAGEB : 15;
  static constexpr int MAX_STAGES = 16;
  static_assert(STAGES >= 2 && STAGES < MAX_STAGES, "stages");
};
__host__ __device__ constexpr int q4_red_bytes(int warps, int rows, int d) {
  return warps * rows * step_red_stride(d) * (int)sizeof(float);
}
constexpr int kQ4TailBytes = 2 * 16 * 8 + 64 + 16 * 8;
template <int D>
constexpr int kQ4BytesMost =
    Q4Cfg<D>::STAGES * Q4Cfg<D>::STAGEB + q4_red_bytes(Q4Cfg<D>::WARPS, kStepRows, D) + kQ4TailBytes + 128;
static_assert(sizeof(StepMisc<8>) <= 64 + 16 * 8, "misc");

template <int D>
__device__ void q4_produce(const StepArgs& a, const Q4Pool& pool, const PagedWork& w, PagedCursor c, PagedSeg g,
                           uint32_t base, uint32_t full, uint32_t empty, const StepWait& wt) {
  using C = Q4Cfg<D>;
  const int lane = threadIdx.x & 31;
  const int shift = a.p.page_shift, ps = 1 << shift;
  int st = 0;
  uint32_t ph = 1, count = 0;
  bool ok = true;
  while (ok && c.next(a.p, w, &g)) {
    const int32_t* row = a.p.page_table + (long long)g.b * a.p.max_pages;
    const int end = g.walk.end();
    const int pages = (end + ps - 1) >> shift;  // of the sequence, as far as the tile sees
    PageIds ids;
    for (int i = 0; i < g.n; ++i) {
      const int tok0 = g.walk.block(g.i0 + i) << kStepShift;
      const int p0 = tok0 >> shift;
      const int valid = end - tok0 < C::KEYS ? end - tok0 : C::KEYS;
      const int npg = ps >= C::KEYS ? 1 : (valid + ps - 1) >> shift;  // at most 8
      ids.cover(row, p0, npg, pages);
      const int page = ids.get(p0 + lane);
      const uint32_t bar = full + 8u * st;
      if (!(ok = __all_sync(0xffffffffu, step_wait(empty + 8u * st, ph, wt, kSiteStepEmpty)))) break;
      const bool mine = lane < npg, good = page >= 0 && page < a.p.num_pages;
      const unsigned bad = __ballot_sync(0xffffffffu, mine && !good);
      const uint32_t dst = base + st * C::STAGEB;
      if (bad) {
        // read as zeros: silu(0) V = 0
        if (lane == 0) atomicOr(a.status, kStatusBadPaged);
        for (int j = 0; j < npg; ++j)
          if (bad >> j & 1u)
            for (int x = 16 * lane; x < pool.tile_bytes; x += 16 * 32)
              asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(dst + j * pool.tile_bytes + x), "r"(0)
                           : "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
      }
      if (lane == 0) mbar_arrive_expect_tx(bar, (uint32_t)((npg - __popc(bad)) * pool.tile_bytes));
      __syncwarp();
      if (mine && good) {
        const int sub = (tok0 & (ps - 1)) >> pool.tile_shift;  // 0 but for pages of more than a block
        bulk_load(dst + lane * pool.tile_bytes,
                  pool.pages + page * pool.page_stride + ((long long)g.h * pool.tiles + sub) * pool.tile_bytes,
                  (uint32_t)pool.tile_bytes, bar);
      }
      ++count;
      if (++st == a.stages) {
        st = 0;
        ph ^= 1u;
      }
    }
  }
  // every copy lands before the CTA ends (as step_produce)
  if (lane == 0) {
    for (int s = 0; s < a.stages; ++s)
      if (count > (uint32_t)s) {
        const uint32_t parity = ((count - 1u - s) / a.stages) & 1u;
        const uint64_t t0 = globaltimer();
        while (!mbar_try_wait(full + 8u * s, parity))
          if (globaltimer() - t0 > 2000000000ull) break;
      }
  }
  __syncwarp();
}

__device__ __forceinline__ uint32_t lds8(uint32_t at) {
  uint32_t x;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(x) : "r"(at) : "memory");
  return x;
}
__device__ __forceinline__ uint32_t lds16(uint32_t at) {
  uint32_t x;
  asm volatile("ld.shared.u16 %0, [%1];" : "=r"(x) : "r"(at) : "memory");
  return x;
}
template <int WORDS>
__device__ __forceinline__ void lds_words(uint32_t at, uint32_t (&w)[WORDS]) {
  if constexpr (WORDS == 1)
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w[0]) : "r"(at) : "memory");
  else if constexpr (WORDS == 2)
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(at) : "memory");
  else
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                 : "r"(at)
                 : "memory");
}

// The key, of 8, of column 2 t + e of a tile of S.
template <int D>
__device__ __forceinline__ int q4_key(int t, int e) {
  return 4 * e + ((t + (D == 128 ? e : 2 * e)) & 3);
}

template <int D, bool CLUSTER>
__device__ void q4_compute(const StepArgs& a, const Q4Pool& pool, const PagedWork& w, PagedCursor c, PagedSeg g,
                           uint32_t base, uint32_t full, uint32_t empty, float* red,
                           StepMisc<Q4Cfg<D>::WARPS>* m, const StepWait& wt) {
  using C = Q4Cfg<D>;
  using T = Q4Tile<D>;
  constexpr int KS = C::KW / 16;            // k16 steps of the P V product
  constexpr int KWORDS = D / 32;            // words of a lane's channels of a key
  constexpr int VWORDS = D >= 64 ? D / 64 : 1;  // of a value: at d = 32 half a word
  constexpr int NT = D / 8;                 // n tiles of O
  constexpr int RS = step_red_stride(D);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g8 = lane >> 2, t4 = lane & 3;
  // bytes of the lane's keys, values and scales in a stage, for each k16 step
  uint32_t k_at[KS], v_at[KS], ks_at[KS], vs_at[KS];
  int key0[KS];  // the step's first key
#pragma unroll
  for (int y = 0; y < KS; ++y) {
    key0[y] = C::KW * warp + 16 * y;
    const int sub = key0[y] >> pool.tile_shift, r = key0[y] & ((1 << pool.tile_shift) - 1);
    const uint32_t tile = base + sub * pool.tile_bytes;
    const int kr = r + q4_key<D>(g8 >> 1, g8 & 1);
    k_at[y] = tile + T::codes(pool.tile_shift, 0, kr) + t4 * (D / 8);
    ks_at[y] = tile + T::scales(pool.tile_shift, 0, kr) + t4 * (D / 4) / kQ4Group;
    v_at[y] = tile + T::codes(pool.tile_shift, 1, r) + g8 * (D / 16);
    vs_at[y] = tile + T::scales(pool.tile_shift, 1, r) + g8 * (D / 8) / kQ4Group;
  }
  const int vk[2] = {q4_key<D>(t4, 0), q4_key<D>(t4, 1)};
  const float2 ha2 = make_float2(a.half_alpha, a.half_alpha);
  int st = 0;
  uint32_t ph = 0;
  // The CTA gave up: go through the items' barriers, but touch no stage (one
  // that was not waited for is not released either) and store nothing.
  bool dead = false;
  StepCut cut0{}, cut1{};  // items shared with earlier, and with later, CTAs
  // test hook: the barrier behind the stages' is never arrived on
  if (a.debug_flags & kDebugUnsignalledWait)
    dead = !__all_sync(0xffffffffu, step_wait(full + 8u * C::MAX_STAGES - 8u, 0, wt, kSiteUnsignalledStep));
  while (c.next(a.p, w, &g)) {
    const int rows = g.walk.rows;
    const bool few = rows <= 8;
    uint32_t qf[D / 16][4];
    {
      const uint16_t* x0 =
          a.q + (long long)(g.seq.q0 + kStepRows * g.qt + g8) * a.q_stride + (long long)g.h * D + t4 * (D / 4);
      const uint16_t* x1 = x0 + 8 * a.q_stride;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const uint4 u = g8 < rows ? load16(x0 + 8 * i) : make_uint4(0u, 0u, 0u, 0u);
        const uint4 v = g8 + 8 < rows ? load16(x1 + 8 * i) : make_uint4(0u, 0u, 0u, 0u);
        qf[2 * i][0] = u.x;
        qf[2 * i][2] = u.y;
        qf[2 * i + 1][0] = u.z;
        qf[2 * i + 1][2] = u.w;
        qf[2 * i][1] = v.x;
        qf[2 * i][3] = v.y;
        qf[2 * i + 1][1] = v.z;
        qf[2 * i + 1][3] = v.w;
      }
    }
    float o[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int j = 0; j < 4; ++j) o[n][j] = 0.f;

    for (int i = 0; i < g.n && !dead; ++i) {
      const int kb = g.walk.block(g.i0 + i) << kStepShift;
      if ((dead = !__all_sync(0xffffffffu, step_wait(full + 8u * st, ph, wt, kSiteStepFull)))) break;
      const uint32_t off = st * C::STAGEB;
      float s[2 * KS][4];
#pragma unroll
      for (int n = 0; n < 2 * KS; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[n][j] = 0.f;
#pragma unroll
      for (int y = 0; y < KS; ++y) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t kw[KWORDS];
          lds_words<KWORDS>(off + k_at[y] + 8 * h * T::CODEB, kw);
          const uint32_t sat = off + ks_at[y] + 8 * h * T::SCALEB;
          const uint32_t j = D == 128 ? lds16(sat) : lds8(sat);
          Q4Scale sc = q4_scale(j & 255u, j & 255u);
#pragma unroll
          for (int x = 0; x < KWORDS; ++x) {
            if (x == 2) sc = q4_scale(j >> 8, j >> 8);
            mma16816(s[2 * y + h], qf[2 * x], q4_pair<0>(kw[x], sc), q4_pair<1>(kw[x], sc));
            mma16816(s[2 * y + h], qf[2 * x + 1], q4_pair<2>(kw[x], sc), q4_pair<3>(kw[x], sc));
          }
        }
      }
      // p = silu(alpha S) = h + h tanh(h), h = alpha S / 2
      const bool masked = kb + C::KEYS > g.walk.p0 + 1 || kb + C::KEYS > g.seq.hist;
      uint32_t hi[KS][4], lo[KS][4];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        if (r == 0 || !few) {
#pragma unroll
          for (int n = 0; n < 2 * KS; ++n) {
            const float2 x = __fmul2_rn(make_float2(s[n][2 * r], s[n][2 * r + 1]), ha2);
            float2 p = __ffma2_rn(x, make_float2(tanh_approx(x.x), tanh_approx(x.y)), x);
            if (masked) {
              const int pos = g.walk.p0 + 8 * r + g8, k0 = kb + key0[n >> 1] + 8 * (n & 1);
              const int x0 = k0 + vk[0], x1 = k0 + vk[1];
              if (!(x0 <= pos && (x0 < g.seq.hist || x0 == pos))) p.x = 0.f;
              if (!(x1 <= pos && (x1 < g.seq.hist || x1 == pos))) p.y = 0.f;
            }
            const uint32_t ph2 = pack_bf16x2(p.x, p.y);
            const float2 rest = __fadd2_rn(
                p, make_float2(-__uint_as_float(ph2 << 16), -__uint_as_float(ph2 & 0xffff0000u)));
            hi[n >> 1][2 * (n & 1) + r] = ph2;
            lo[n >> 1][2 * (n & 1) + r] = pack_bf16x2(rest.x, rest.y);
          }
        } else {
          // rows 8 .. 15 of the operand: the second terms of rows 0 .. 7
#pragma unroll
          for (int n = 0; n < 2 * KS; ++n) hi[n >> 1][2 * (n & 1) + 1] = lo[n >> 1][2 * (n & 1)];
        }
      }
#pragma unroll
      for (int y = 0; y < KS; ++y) {
        // four keys: vw[h][e] is key 8 h + vk[e] of the step
        uint32_t vw[2][2][VWORDS];
        Q4Scale sc[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t j[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint32_t at = off + v_at[y] + (8 * h + vk[e]) * T::CODEB;
            if constexpr (D == 32)
              vw[h][e][0] = lds16(at);
            else
              lds_words<VWORDS>(at, vw[h][e]);
            j[e] = lds8(off + vs_at[y] + (8 * h + vk[e]) * T::SCALEB);
          }
          sc[h] = q4_scale(j[0], j[1]);
        }
#pragma unroll
        for (int x = 0; x < VWORDS; ++x) {
#pragma unroll
          for (int half = 0; half < (D == 32 ? 1 : 2); ++half) {
            uint32_t u[2];  // the keys' even, then odd, channels side by side
#pragma unroll
            for (int h = 0; h < 2; ++h) u[h] = __byte_perm(vw[h][0][x], vw[h][1][x], half ? 0x7632 : 0x5410);
            uint32_t b[4][2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              b[0][h] = q4_pair<0>(u[h], sc[h]);
              b[1][h] = q4_pair<1>(u[h], sc[h]);
              b[2][h] = q4_pair<2>(u[h], sc[h]);
              b[3][h] = q4_pair<3>(u[h], sc[h]);
            }
#pragma unroll
            for (int n = 0; n < 4; ++n) {
              float(&acc)[4] = o[D == 32 ? n : 8 * x + 2 * n + half];
              mma16816(acc, hi[y], b[n][0], b[n][1]);
            }
            if (!few) {
#pragma unroll
              for (int n = 0; n < 4; ++n) {
                float(&acc)[4] = o[D == 32 ? n : 8 * x + 2 * n + half];
                mma16816(acc, lo[y], b[n][0], b[n][1]);
              }
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(empty + 8u * st);
      if (++st == a.stages) {
        st = 0;
        ph ^= 1u;
      }
    }

    // the warps' sums over their keys, then out or this CTA's part.  Columns
    // 2 t4 + e of O's n tiles are D / 8 consecutive channels.
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int row = 8 * r + g8;
      if (row < rows) {
        float* dst = red + (warp * a.red_rows + row) * RS + t4 * (D / 4);
        auto val = [&](int n, int e) { return few ? o[n][e] + o[n][2 + e] : o[n][2 * r + e]; };
        if constexpr (D == 32) {
#pragma unroll
          for (int n = 0; n < 4; n += 2)
            *reinterpret_cast<float4*>(dst + 2 * n) =
                make_float4(val(n, 0), val(n, 1), val(n + 1, 0), val(n + 1, 1));
        } else {
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int n = 0; n < NT; n += 4)
              *reinterpret_cast<float4*>(dst + e * NT + n) =
                  make_float4(val(n, e), val(n + 1, e), val(n + 2, e), val(n + 3, e));
        }
      }
    }
    step_barrier<C::WARPS>();
    if constexpr (CLUSTER) {
      for (int x = 4 * threadIdx.x; x < rows * D; x += 4 * 32 * C::WARPS) {
        float* at = red + (x / D) * RS + x % D;
        float4 v = *reinterpret_cast<const float4*>(at);
#pragma unroll
        for (int i = 1; i < C::WARPS; ++i)
          add4(v, *reinterpret_cast<const float4*>(at + i * a.red_rows * RS));
        *reinterpret_cast<float4*>(at) = v;
      }
      return;  // one segment a CTA
    }
    // one answer for the warp, whose lanes meet again in the next item's waits:
    // the copying warp may give up between two lanes' reads
    dead = __any_sync(0xffffffffu, *static_cast<volatile int*>(&m->abort_flag) != 0);
    uint16_t* out = a.out + ((long long)(g.seq.q0 + kStepRows * g.qt) * w.heads + g.h) * D;
    const bool before = g.c0 != (int)blockIdx.x;
    float* part = step_part<D>(a, blockIdx.x, !before);
    for (int x = 4 * threadIdx.x; x < rows * D; x += 4 * 32 * C::WARPS) {
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int i = 0; i < C::WARPS; ++i)
        add4(v, *reinterpret_cast<const float4*>(red + (i * a.red_rows + x / D) * RS + x % D));
      if (dead) continue;
      if (g.parts == 1)
        step_store<D>(out, w.heads, x, v, a.inv_n);
      else
        __stcg(reinterpret_cast<float4*>(part + x), v);
    }
    if (g.parts > 1) {
      const StepCut cut{out, rows, g.c0, g.parts};
      if (before)
        cut0 = cut;
      else
        cut1 = cut;
    }
    step_barrier<C::WARPS>();  // red is free for the next item
  }
  step_join<D, C::WARPS>(a, w, m, cut0, cut1, dead);
}

template <int D, bool CLUSTER>
__global__ void __launch_bounds__(Q4Cfg<D>::THREADS, Q4Cfg<D>::PER_SM)
    step_q4_kernel(const StepArgs a, const Q4Pool pool) {
  using C = Q4Cfg<D>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 127u) & ~127u;
  uint8_t* tail = smem_raw + (base - raw) + a.stages * C::STAGEB;
  float* red = reinterpret_cast<float*>(tail);
  uint8_t* after = tail + q4_red_bytes(C::WARPS, a.red_rows, D);
  const uint32_t full = smem_u32(after), empty = full + 8u * C::MAX_STAGES;
  auto* m = reinterpret_cast<StepMisc<C::WARPS>*>(after + 2 * C::MAX_STAGES * 8);
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x < a.stages) {
    mbar_init(full + 8u * threadIdx.x, 1);
    mbar_init(empty + 8u * threadIdx.x, C::WARPS);
    if (threadIdx.x == 0) {
      m->abort_flag = 0;
      mbar_init(full + 8u * C::MAX_STAGES - 8u, 1);  // for the test hook alone: a.stages < MAX_STAGES
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  after_previous_kernel();
  PagedWork w = a.w;
  PagedCursor c;
  PagedSeg g;
  int rank = 0;
  if constexpr (CLUSTER) {
    rank = (int)blockIdx.x % kStepCluster;
    if (!step_cluster_share(a, rank, &w, &c, &g)) return;  // the same for the whole cluster
    if (c.u1 == 0)  // no block of its own: its sums are zero
      for (int x = threadIdx.x; x < a.red_rows * step_red_stride(D); x += C::THREADS) red[x] = 0.f;
    __syncthreads();
  } else {
    if (!paged_locate<C::WARPS + 1, false>(a.p, &w, &m->start, a.status, &c, &g)) return;
  }
  const StepWait wt{a.timeout_ns, &m->abort_flag, a.status};
  if (warp == C::WARPS)
    q4_produce<D>(a, pool, w, c, g, base, full, empty, wt);
  else
    q4_compute<D, CLUSTER>(a, pool, w, c, g, base, full, empty, red, m, wt);
  if constexpr (CLUSTER) step_cluster_join<D, C::THREADS>(a, g, rank, red, &m->abort_flag);
}

template <int D>
cudaError_t q4_prepare() {
  static DeviceOnce once;
  return once.run([] {
    const cudaError_t e = cudaFuncSetAttribute(
        step_q4_kernel<D, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, kQ4BytesMost<D>);
    if (e != cudaSuccess) return e;
    return cudaFuncSetAttribute(step_q4_kernel<D, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                kQ4BytesMost<D>);
  });
}

template <int D>
cudaError_t clusters_q4(int* n) {
  const cudaError_t e = q4_prepare<D>();
  if (e != cudaSuccess) return e;
  return clusters_at_once(step_q4_kernel<D, true>, Q4Cfg<D>::THREADS, kQ4BytesMost<D>, n);
}

template <int D>
cudaError_t launch_step_q4_d(const Q4Pool& pool, long long most, bool clusters, StepArgs a, int sms,
                             cudaStream_t stream) {
  using C = Q4Cfg<D>;
  a.stages = C::STAGES;
  const int bytes = a.stages * C::STAGEB + q4_red_bytes(C::WARPS, a.red_rows, D) + kQ4TailBytes + 128;
  const cudaError_t e = q4_prepare<D>();
  if (e != cudaSuccess) return e;
  if (clusters)
    return launch_after_in_clusters(kStepCluster, step_q4_kernel<D, true>,
                                    kStepCluster * a.w.tiles * a.p.batch * a.w.heads, C::THREADS, bytes,
                                    stream, a, pool);
  const int grid = (int)std::min<long long>((long long)C::PER_SM * sms, most);
  return launch_after(step_q4_kernel<D, false>, grid, C::THREADS, bytes, stream, a, pool);
}

template <int D>
cudaError_t launch_append_q4_d(const Q4Pool& pool, const AppendArgs& a, cudaStream_t stream) {
  const int grid = (int)(a.check_ctas + q4_blocks<D>(a.p.rows, a.heads));
  return launch_after(append_q4_kernel<D>, grid, kQ4Threads, 0, stream, a, pool);
}

template <int D>
cudaError_t launch_read_q4_d(const Q4Pool& pool, const ReadArgs& a, cudaStream_t stream) {
  const int grid = (int)(a.check_ctas + q4_blocks<D>(a.p.rows, a.heads));
  return launch_after(read_q4_kernel<D>, grid, kQ4Threads, 0, stream, a, pool);
}

}  // namespace

cudaError_t launch_append_q4(const Q4Pool& pool, const AppendArgs& a, cudaStream_t stream) {
  switch (a.d) {
    case 32: return launch_append_q4_d<32>(pool, a, stream);
    case 64: return launch_append_q4_d<64>(pool, a, stream);
    default: return launch_append_q4_d<128>(pool, a, stream);
  }
}

cudaError_t launch_read_q4(const Q4Pool& pool, const ReadArgs& a, cudaStream_t stream) {
  switch (a.d) {
    case 32: return launch_read_q4_d<32>(pool, a, stream);
    case 64: return launch_read_q4_d<64>(pool, a, stream);
    default: return launch_read_q4_d<128>(pool, a, stream);
  }
}

cudaError_t launch_step_q4(int d, const Q4Pool& pool, long long most, bool clusters, const StepArgs& a,
                           int sms, cudaStream_t stream) {
  switch (d) {
    case 32: return launch_step_q4_d<32>(pool, most, clusters, a, sms, stream);
    case 64: return launch_step_q4_d<64>(pool, most, clusters, a, sms, stream);
    default: return launch_step_q4_d<128>(pool, most, clusters, a, sms, stream);
  }
}

cudaError_t step_clusters_q4(int d, int* n) {
  switch (d) {
    case 32: return clusters_q4<32>(n);
    case 64: return clusters_q4<64>(n);
    default: return clusters_q4<128>(n);
  }
}

}  // namespace hstu
