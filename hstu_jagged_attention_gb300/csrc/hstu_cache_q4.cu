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
// Accesses in flight, each to whole rows: of the append, which has three rows,
// the next head's, and the rotation's angles in registers, and of the reading.
// 65,536 tokens of 4 heads of 64: append 33.5 us with one, 33.8 with two;
// reading 19.6 with one, 17.8 with two, 18.7 with four.
constexpr int kQ4AppendIter = 1, kQ4ReadIter = 2;
// Warps an SM below which a warp takes fewer heads: 6,700 tokens of 4 heads of
// 128 are appended in 6.8 us with 8 and 16, 9.3 with 24 (three heads and one),
// and read in 6.9, 5.5 and 6.2 with 8, 16 and 24 (four, two and one); 65,536 of
// 4 heads of 64 are appended in 33.5 us, 56 with a head a warp.
constexpr int kQ4Warps = 16;

// How a warp of the append and of the reading works: a lane has 8 channels (a
// word of codes) of one head, D / 8 neighbouring lanes a token, so that each
// access of the warp is to whole rows one behind the other, and ITER such
// accesses are in flight.  The first lanes look the warp's tokens up, a token
// each, and hand out what they found.
template <int D, int ITER>
struct Q4Rows {
  static constexpr int LANES = D / 8;         // of a token
  static constexpr int TOKENS = 32 / LANES;   // of an access
  static constexpr int ALL = TOKENS * ITER;   // of a warp
  static_assert(ALL <= 32, "a lane a token");
};
// Warps that take all the tokens' heads `step` at a time, and the CTAs of them.
template <int D, int ITER>
long long q4_blocks(long long rows, int heads, int step) {
  constexpr int ALL = Q4Rows<D, ITER>::ALL;
  return ((rows + ALL - 1) / ALL * ((heads + step - 1) / step) * 32 + kQ4Threads - 1) / kQ4Threads;
}
// A warp looks its tokens up once for all the heads it takes, and has the next
// head's rows in flight while it works on one's; but it takes only as many as
// leave kQ4Warps an SM.
template <int D, int ITER>
int q4_head_step(long long rows, int heads, int sms) {
  constexpr int ALL = Q4Rows<D, ITER>::ALL;
  const long long warps = (rows + ALL - 1) / ALL * heads;
  return (int)std::max<long long>(1, std::min<long long>(heads, warps / ((long long)kQ4Warps * sms)));
}

// The first CTAs check a sequence a thread: one that contradicts itself may
// have no row.
unsigned q4_check_ctas(const PagedView& p) { return ((unsigned)p.batch + kQ4Threads - 1) / kQ4Threads; }
__device__ __forceinline__ bool q4_checks(const PagedView& p, unsigned check_ctas, unsigned* status) {
  if (blockIdx.x >= check_ctas) return false;
  const long long b = (long long)blockIdx.x * kQ4Threads + threadIdx.x;
  PagedSeq s;
  if (b < p.batch && !paged_seq(p, (int)b, &s)) atomicOr(status, kStatusBadPaged);
  return true;
}

// A token's place: its tile in the first head, its row there (-1: it has none, -2: its page is
// out of range), and the position it is turned to.
struct Q4Place {
  long long tile;  // bytes
  int row, turned_at;
};
__device__ __forceinline__ Q4Place q4_place(const PagedView& p, const Q4Pool& pool, long long t) {
  Q4Place x{0, -1, 0};
  PagedSeq s;
  if (t >= p.rows) return x;
  const int b = paged_find(p, (int)t);
  if (b < 0 || !paged_seq(p, b, &s)) return x;  // of no sequence, or of one that is reported
  const int pos = s.kv - s.qn + ((int)t - s.q0);
  const long long slot = paged_slot(p, b, pos);
  x.turned_at = pos < s.hist ? pos : s.hist;  // a candidate stands right behind the history
  x.row = -2;
  if (slot < 0) return x;
  const int in_page = (int)(slot & ((1 << p.page_shift) - 1));
  x.row = in_page & ((1 << pool.tile_shift) - 1);
  x.tile = (slot >> p.page_shift) * pool.page_stride + (long long)(in_page >> pool.tile_shift) * pool.tile_bytes;
  return x;
}
__device__ __forceinline__ Q4Place q4_place_of(const Q4Place& mine, int lane) {
  return Q4Place{__shfl_sync(0xffffffffu, mine.tile, lane), __shfl_sync(0xffffffffu, mine.row, lane),
                 __shfl_sync(0xffffffffu, mine.turned_at, lane)};
}

__device__ __forceinline__ uint4 load16(const uint16_t* p) { return *reinterpret_cast<const uint4*>(p); }

// The angles of a lane's 8 channels: cosines, and the sines that its partner's
// channels are multiplied with (pairs of channels: 4 angles, halves: 8).
struct Q4Angles {
  float cs[8], sn[8];
};
// This lane's channels x, of c .. c + 7 of the head, rotated if c < rot.  Where
// the channels turn in halves the partner's are rot / 16 lanes away.  The
// products are rounded one by one, as a plain form does: what is quantised then
// is the same number, not one beside it across a border.  (Products and sums of
// two floats at once come out fused.)  Whole-warp call.
__device__ __forceinline__ uint4 q4_turn(const uint4& x, const Q4Angles& g, int c, int rot, bool pairs) {
  F8 a = unpack8(x);
  if (pairs) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float u = a.f[2 * i], v = a.f[2 * i + 1];
      a.f[2 * i] = __fsub_rn(__fmul_rn(u, g.cs[i]), __fmul_rn(v, g.sn[i]));
      a.f[2 * i + 1] = __fadd_rn(__fmul_rn(v, g.cs[i]), __fmul_rn(u, g.sn[i]));
    }
  } else {
    const int other = (threadIdx.x & 31) + (c >= rot ? 0 : c < rot >> 1 ? rot >> 4 : -(rot >> 4));
    const uint4 y = make_uint4(__shfl_sync(0xffffffffu, x.x, other), __shfl_sync(0xffffffffu, x.y, other),
                               __shfl_sync(0xffffffffu, x.z, other), __shfl_sync(0xffffffffu, x.w, other));
    const F8 b = unpack8(y);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      a.f[i] = __fadd_rn(__fmul_rn(a.f[i], g.cs[i]), __fmul_rn(b.f[i], g.sn[i]));
  }
  return c < rot ? pack8(a) : x;
}

// 65,536 tokens of 4 heads of 64 with their queries, rotated, take 33.5 us (153
// MB, 4.6 TB/s).  Bound by instructions and memory alike: a warp executes 398 for
// its lanes' 8 channels of k, v and q (26.1 M, whose issue alone takes 21 us; 157
// of them on the ALU pipe, 55% busy), the issue slots are 70% busy, and the bytes
// take 22.6 us.
template <int D>
__global__ void __launch_bounds__(kQ4Threads)
    append_q4_kernel(const AppendArgs a, const Q4Pool pool, const int head_step) {
  using T = Q4Tile<D>;
  constexpr int ITER = kQ4AppendIter;
  using R = Q4Rows<D, ITER>;
  after_previous_kernel();
  if (q4_checks(a.p, a.check_ctas, a.status)) return;
  const int lane = threadIdx.x & 31;
  const long long w = ((long long)(blockIdx.x - a.check_ctas) * kQ4Threads + threadIdx.x) >> 5;
  const int parts = (a.heads + head_step - 1) / head_step;
  const long long t0 = w / parts * R::ALL;
  if (t0 >= a.p.rows) return;  // the same for the warp
  int h = (int)(w % parts) * head_step;
  const int h1 = h + head_step < a.heads ? h + head_step : a.heads;
  const int c = 8 * (lane % R::LANES);  // the lane's channels of a head
  const long long mine_t = t0 + lane / R::LANES;
  struct Rows {
    uint4 k[ITER], v[ITER], q[ITER];
  };
  auto load = [&](Rows& x, int head) {
    const long long at = (long long)head * D + c;
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
      const long long t = mine_t + i * R::TOKENS;
      x.k[i] = x.v[i] = x.q[i] = make_uint4(0u, 0u, 0u, 0u);
      if (t < a.p.rows) {
        x.k[i] = load16(a.k + t * a.k_stride + at);
        x.v[i] = load16(a.v + t * a.v_stride + at);
        if (a.q) x.q[i] = load16(a.q + t * a.q_stride + at);
      }
    }
  };
  Rows next;
  load(next, h);
  Q4Place mine{0, -1, 0}, place[ITER];
  if (lane < R::ALL) {
    mine = q4_place(a.p, pool, t0 + lane);
    if (mine.row == -2 || (mine.row >= 0 && a.table && mine.turned_at >= a.positions)) {
      atomicOr(a.status, kStatusBadPaged);  // dropped
      mine.row = -1;
    }
  }
  Q4Angles angles[ITER];
  const int half = a.rot >> 1;
#pragma unroll
  for (int i = 0; i < ITER; ++i) {
    place[i] = q4_place_of(mine, i * R::TOKENS + lane / R::LANES);
    float4 cs[2], sn[2];
    cs[0] = cs[1] = sn[0] = sn[1] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (a.table && place[i].row >= 0 && c < a.rot) {
      const float* tab =
          a.table + (long long)place[i].turned_at * a.rot + (a.pairs ? c >> 1 : c < half ? c : c - half);
      cs[0] = __ldg(reinterpret_cast<const float4*>(tab));
      sn[0] = __ldg(reinterpret_cast<const float4*>(tab + half));
      if (!a.pairs) {
        cs[1] = __ldg(reinterpret_cast<const float4*>(tab) + 1);
        sn[1] = __ldg(reinterpret_cast<const float4*>(tab + half) + 1);
      }
    }
    const float sign = !a.pairs && c < half ? -1.f : 1.f;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float cc[4] = {cs[k].x, cs[k].y, cs[k].z, cs[k].w}, ss[4] = {sn[k].x, sn[k].y, sn[k].z, sn[k].w};
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        angles[i].cs[4 * k + m] = cc[m];
        angles[i].sn[4 * k + m] = sign * ss[m];
      }
    }
  }
#pragma unroll 1
  for (; h < h1; ++h) {
    Rows x = next;
    if (h + 1 < h1) load(next, h + 1);
    const long long head = (long long)h * pool.tiles * pool.tile_bytes;
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
      if (a.table) {
        x.k[i] = q4_turn(x.k[i], angles[i], c, a.rot, a.pairs);
        if (a.q) x.q[i] = q4_turn(x.q[i], angles[i], c, a.rot, a.pairs);
      }
      uint32_t kj, vj;
      const uint32_t kc = q4_quantise(x.k[i], &kj), vc = q4_quantise(x.v[i], &vj);
      const int row = place[i].row;
      if (row >= 0) {
        uint8_t* tile = pool.pages + place[i].tile + head;
        *reinterpret_cast<uint32_t*>(tile + T::codes(pool.tile_shift, 0, row) + c / 2) = kc;
        *reinterpret_cast<uint32_t*>(tile + T::codes(pool.tile_shift, 1, row) + c / 2) = vc;
        if (lane & 1)
          tile[T::scales(pool.tile_shift, 1, row) + c / kQ4Group] = (uint8_t)vj;
        else
          tile[T::scales(pool.tile_shift, 0, row) + c / kQ4Group] = (uint8_t)kj;
        if (a.q)
          *reinterpret_cast<uint4*>(a.q_out + ((mine_t + i * R::TOKENS) * a.heads + h) * D + c) = x.q[i];
      }
    }
  }
}

// 65,536 tokens of 4 heads of 64 take 17.8 us (86 MB, 4.8 TB/s), 156,000 of 32
// histories 38.1 (205 MB, 5.4 TB/s, 79% of a copy's rate).  Bound by memory: 136
// instructions for a lane's 8 channels of k and v keep 58% of the issue slots
// busy, and what a warp waits for most are its loads (40% of its time).
template <int D>
__global__ void __launch_bounds__(kQ4Threads)
    read_q4_kernel(const ReadArgs a, const Q4Pool pool, const int head_step) {
  using T = Q4Tile<D>;
  constexpr int ITER = kQ4ReadIter;
  using R = Q4Rows<D, ITER>;
  after_previous_kernel();
  if (q4_checks(a.p, a.check_ctas, a.status)) return;
  const int lane = threadIdx.x & 31;
  const long long w = ((long long)(blockIdx.x - a.check_ctas) * kQ4Threads + threadIdx.x) >> 5;
  const int parts = (a.heads + head_step - 1) / head_step;
  const long long t0 = w / parts * R::ALL;
  if (t0 >= a.p.rows) return;  // the same for the warp
  int h = (int)(w % parts) * head_step;
  const int h1 = h + head_step < a.heads ? h + head_step : a.heads;
  const int c = 8 * (lane % R::LANES);
  Q4Place mine{0, -1, 0}, place[ITER];
  if (lane < R::ALL) {
    mine = q4_place(a.p, pool, t0 + lane);
    if (mine.row == -2) atomicOr(a.status, kStatusBadPaged);  // read as zeros
  }
#pragma unroll
  for (int i = 0; i < ITER; ++i) place[i] = q4_place_of(mine, i * R::TOKENS + lane / R::LANES);
  struct Codes {
    uint32_t kc[ITER], vc[ITER], kj[ITER], vj[ITER];
  };
  // coherent loads: an append may write the pool until the wait above returns
  auto load = [&](Codes& x, int head) {
    const long long off = (long long)head * pool.tiles * pool.tile_bytes;
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
      x.kc[i] = x.vc[i] = x.kj[i] = x.vj[i] = 0;
      const int row = place[i].row;
      if (row >= 0) {
        const uint8_t* tile = pool.pages + place[i].tile + off;
        x.kc[i] = *reinterpret_cast<const uint32_t*>(tile + T::codes(pool.tile_shift, 0, row) + c / 2);
        x.vc[i] = *reinterpret_cast<const uint32_t*>(tile + T::codes(pool.tile_shift, 1, row) + c / 2);
        x.kj[i] = tile[T::scales(pool.tile_shift, 0, row) + c / kQ4Group];
        x.vj[i] = tile[T::scales(pool.tile_shift, 1, row) + c / kQ4Group];
      }
    }
  };
  Codes next;
  load(next, h);
#pragma unroll 1
  for (; h < h1; ++h) {
    const Codes x = next;
    if (h + 1 < h1) load(next, h + 1);
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
      if (place[i].row == -1) continue;
      const long long t = t0 + i * R::TOKENS + lane / R::LANES, at = (long long)h * D + c;
      *reinterpret_cast<uint4*>(a.k + t * a.k_stride + at) = q4_word(x.kc[i], q4_scale(x.kj[i]));
      *reinterpret_cast<uint4*>(a.v + t * a.v_stride + at) = q4_word(x.vc[i], q4_scale(x.vj[i]));
    }
  }
}

// ------------------------------------------------ attention of a few tokens
// As the bf16 cache's kernel of 16-row tiles (hstu_cache.cu): the last warp
// copies blocks of 128 keys with their values into a ring of shared-memory
// stages, one bulk copy a page, and the others take a part of the keys each.
// The codes become the products' A operands (16 keys, or 16 channels) in
// registers, and the few new tokens are their 8 columns, so that no product's
// rows are padding:
//   S^T = K Q^T: a lane's operand of key m is channels 2 t .. and 2 t + 8 .. of
//     every 16; a sum over channels may take them in any order, so lane t has
//     the D / 4 consecutive channels whose codes it loads with one access, and
//     Q's operand the same ones;
//   O^T += V^T P^T: lane n's operand is channels n and n + 8 of keys 2 t, 2 t +
//     1, 2 t + 8 and 2 t + 9.  It loads D / 8 consecutive channels of its four
//     keys, and one byte permutation of two keys' words puts the keys side by
//     side.  Which channel a row of O^T is, and which key a row of S^T, is
//     free, as long as P^T's rows are V^T's columns: key 8 a + 4 e + (t + 2 e)
//     % 4 for row 8 a + 2 t + e lets neither load meet a bank twice (at d = 128,
//     (t + e) % 4: K's do not, V's meet two);
//   P^T's operand is S^T's result transposed: one movmatrix a 8 x 8 tile.
// p is split into two bf16 terms.  TOKENS: what a tile holds, 4, 8 or 16 (two
// groups of columns).  With 4, columns 4 .. 7 are the same tokens' and take the
// second terms: one product for both.
// Keys past a row's last are masked by a select on p; whatever bytes lie
// there, as codes they are finite, and so add nothing.
// Bound by the latency of what a warp does one after the other, which the three
// warps a scheduler has do not cover, and by the way in and out: one token for
// 512 sequences (log-normal lengths, 2 heads of 64, 59 MB) takes 27.4 us, 4 of
// them until the first codes are there and 1.5 to join the cut items.  Issuing
// its 15.5 M instructions takes 12.3 us, the ALU pipe's share of them, 7.4 M at
// half rate, 11.7; the slots are 54% busy.  For each instruction that it issues
// (ncu, in issue cycles) a warp is ready but not chosen for 0.8, and waits 1.2 for
// the one before it, 0.8 for global memory, 0.6 for a pipe, 0.5 for the other
// warps, 0.4 for instructions and 0.3 for shared memory.  Four warps of 32 keys
// and three CTAs an SM: 29.3 us when two took 31.6, four (96 registers a thread)
// 31.3, and two of eight warps of 16 keys 34.6; at d = 128 registers allow two.
template <int D>
struct Q4Cfg {
  static constexpr int WARPS = 4;
  static constexpr int THREADS = 32 * (WARPS + 1);
  static constexpr int KEYS = kStepKeys;
  static constexpr int KW = KEYS / WARPS;
  static constexpr int STAGEB = KEYS * q4_token_bytes(D);
  static constexpr int PER_SM = D == 128 ? 2 : 3;
  // 16-key steps of a warp in one piece of code (with one: 28.9 us)
  static constexpr int UNROLL = 2;
  static constexpr int RING = 128 * 1024 / PER_SM;
  static constexpr int STAGES = RING / STAGEB < 15 ? RING / STAGEB : 15;
  static constexpr int MAX_STAGES = 16;
  static_assert(STAGES >= 2 && STAGES < MAX_STAGES, "stages");
  static_assert(PER_SM <= kStepPerSm, "the workspace's parts");
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

// Plain loads and a product that is not volatile, so that the compiler may move
// them within a block (not across its barriers, which clobber memory).
template <int WORDS>
__device__ __forceinline__ void lds_words(const uint8_t* at, uint32_t (&w)[WORDS]) {
  if constexpr (WORDS == 1) {
    w[0] = *reinterpret_cast<const uint32_t*>(at);
  } else if constexpr (WORDS == 2) {
    const uint2 x = *reinterpret_cast<const uint2*>(at);
    w[0] = x.x;
    w[1] = x.y;
  } else {
    const uint4 x = *reinterpret_cast<const uint4*>(at);
    w[0] = x.x;
    w[1] = x.y;
    w[2] = x.z;
    w[3] = x.w;
  }
}
__device__ __forceinline__ uint32_t lds16(const uint8_t* at) { return *reinterpret_cast<const uint16_t*>(at); }
// d = A B, and c += A B
__device__ __forceinline__ void q4_mma_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void q4_mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// An 8 x 8 tile of 16-bit values, two of a row a lane, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// The key, of 8, of row 2 t + e of a tile of S^T.
template <int D>
__device__ __forceinline__ int q4_key(int t, int e) {
  return 4 * e + ((t + (D == 128 ? e : 2 * e)) & 3);
}

template <int D, int TOKENS, bool CLUSTER>
__device__ void q4_compute(const StepArgs& a, const Q4Pool& pool, const PagedWork& w, PagedCursor c, PagedSeg g,
                           const uint8_t* ring, uint32_t full, uint32_t empty, float* red,
                           StepMisc<Q4Cfg<D>::WARPS>* m, const StepWait& wt) {
  using C = Q4Cfg<D>;
  using T = Q4Tile<D>;
  constexpr int G = TOKENS == 16 ? 2 : 1;       // groups of 8 columns
  constexpr bool both = TOKENS == 4;            // columns 4 .. 7: the second terms of tokens 0 .. 3
  constexpr int KS = C::KW / 16;                // 16-key steps of a block
  constexpr int KWORDS = D / 32;                // words of a lane's channels of a key
  constexpr int VWORDS = D >= 64 ? D / 64 : 1;  // of a value: at d = 32 half a word
  constexpr int MT = D / 16;                    // tiles of O^T
  constexpr int RS = step_red_stride(D);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g8 = lane >> 2, t4 = lane & 3;
  // the lane's keys, values and scales in a stage, for its first 16 keys, and
  // how far the next 16's are: in the same tile, or the next one
  const int vk[2] = {q4_key<D>(t4, 0), q4_key<D>(t4, 1)};
  const int kk = q4_key<D>(g8 >> 1, g8 & 1);
  static_assert(KS <= 2, "two steps are in one tile, or in two");
  const int row0 = (C::KW * warp) & ((1 << pool.tile_shift) - 1);
  const uint8_t* tile = ring + ((C::KW * warp) >> pool.tile_shift) * pool.tile_bytes;
  const bool apart = pool.tile_shift == 4;
  const int codes_step = apart ? pool.tile_bytes : 16 * T::CODEB;
  const int scales_step = apart ? pool.tile_bytes : 16 * T::SCALEB;
  const uint8_t* k_at = tile + T::codes(pool.tile_shift, 0, row0 + kk) + t4 * (D / 8);
  const uint8_t* ks_at = tile + T::scales(pool.tile_shift, 0, row0 + kk) + t4 * (D / 4) / kQ4Group;
  const uint8_t *v_at[2], *vs_at[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    v_at[e] = tile + T::codes(pool.tile_shift, 1, row0 + vk[e]) + g8 * (D / 16);
    vs_at[e] = tile + T::scales(pool.tile_shift, 1, row0 + vk[e]) + g8 * (D / 8) / kQ4Group;
  }
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
    uint32_t qf[G][MT][2];
#pragma unroll
    for (int u = 0; u < G; ++u) {
      const int row = both ? (g8 & 3) : 8 * u + g8;
      const uint16_t* x =
          a.q + (long long)(g.seq.q0 + w.tile_rows * g.qt + row) * a.q_stride + (long long)g.h * D + t4 * (D / 4);
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const uint4 v = row < rows ? load16(x + 8 * i) : make_uint4(0u, 0u, 0u, 0u);
        qf[u][2 * i][0] = v.x;
        qf[u][2 * i][1] = v.y;
        qf[u][2 * i + 1][0] = v.z;
        qf[u][2 * i + 1][1] = v.w;
      }
    }
    float o[G][MT][4];
#pragma unroll
    for (int u = 0; u < G; ++u)
#pragma unroll
      for (int n = 0; n < MT; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[u][n][j] = 0.f;

    for (int i = 0; i < g.n && !dead; ++i) {
      const int kb = g.walk.block(g.i0 + i) << kStepShift;
      if ((dead = !__all_sync(0xffffffffu, step_wait(full + 8u * st, ph, wt, kSiteStepFull)))) break;
      const bool masked = kb + C::KEYS > g.walk.p0 + 1 || kb + C::KEYS > g.seq.hist;
#pragma unroll C::UNROLL
      for (int y = 0; y < KS; ++y) {
        const uint32_t off = st * C::STAGEB + y * codes_step, off_sc = st * C::STAGEB + y * scales_step;
        float s[G][4];
        {
          uint32_t kw[2][KWORDS], j[2];  // keys kk and 8 + kk
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            lds_words<KWORDS>(k_at + off + 8 * h * T::CODEB, kw[h]);
            const uint8_t* sat = ks_at + off_sc + 8 * h * T::SCALEB;
            j[h] = D == 128 ? lds16(sat) : *sat;
          }
          Q4Scale s0 = q4_scale(j[0] & 255u), s1 = q4_scale(j[1] & 255u);
#pragma unroll
          for (int x = 0; x < KWORDS; ++x) {
            if (x == 2) {
              s0 = q4_scale(j[0] >> 8);
              s1 = q4_scale(j[1] >> 8);
            }
            const uint32_t a0[4] = {q4_pair<0>(kw[0][x], s0), q4_pair<0>(kw[1][x], s1), q4_pair<1>(kw[0][x], s0),
                                    q4_pair<1>(kw[1][x], s1)};
            const uint32_t a1[4] = {q4_pair<2>(kw[0][x], s0), q4_pair<2>(kw[1][x], s1), q4_pair<3>(kw[0][x], s0),
                                    q4_pair<3>(kw[1][x], s1)};
#pragma unroll
            for (int u = 0; u < G; ++u) {
              if (x == 0)
                q4_mma_first(s[u], a0, qf[u][0][0], qf[u][0][1]);
              else
                q4_mma(s[u], a0, qf[u][2 * x][0], qf[u][2 * x][1]);
              q4_mma(s[u], a1, qf[u][2 * x + 1][0], qf[u][2 * x + 1][1]);
            }
          }
        }
        // p = silu(alpha S) = h + h tanh(h), h = alpha S / 2
        float2 p[G][2];
#pragma unroll
        for (int u = 0; u < G; ++u)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float2 x = __fmul2_rn(make_float2(s[u][2 * h], s[u][2 * h + 1]), ha2);
            p[u][h] = __ffma2_rn(x, make_float2(tanh_approx(x.x), tanh_approx(x.y)), x);
          }
        if (masked) {
          const int key0 = kb + C::KW * warp + 16 * y + kk;
#pragma unroll
          for (int u = 0; u < G; ++u)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int pos = g.walk.p0 + (both ? 2 * (t4 & 1) : 8 * u + 2 * t4), key = key0 + 8 * h;
              if (!(key <= pos && (key < g.seq.hist || key == pos))) p[u][h].x = 0.f;
              if (!(key <= pos + 1 && (key < g.seq.hist || key == pos + 1))) p[u][h].y = 0.f;
            }
        }
        uint32_t hi[G][2], lo[G][2];
#pragma unroll
        for (int u = 0; u < G; ++u)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t ph2 = pack_bf16x2(p[u][h].x, p[u][h].y);
            const float2 rest = __fadd2_rn(
                p[u][h], make_float2(-__uint_as_float(ph2 << 16), -__uint_as_float(ph2 & 0xffff0000u)));
            const uint32_t pl2 = pack_bf16x2(rest.x, rest.y);
            hi[u][h] = transpose8(both && t4 >= 2 ? pl2 : ph2);
            if constexpr (!both) lo[u][h] = transpose8(pl2);
          }
        // four keys: vw[h][e] is key 8 h + vk[e] of the step
        uint32_t vw[2][2][VWORDS];
        Q4Scale sc[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t j[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint8_t* at = v_at[e] + off + 8 * h * T::CODEB;
            if constexpr (D == 32)
              vw[h][e][0] = lds16(at);
            else
              lds_words<VWORDS>(at, vw[h][e]);
            j[e] = vs_at[e][off_sc + 8 * h * T::SCALEB];
          }
          sc[h] = q4_scale(j[0], j[1]);
        }
#pragma unroll
        for (int x = 0; x < VWORDS; ++x) {
          uint32_t b[4][4];  // operands of four (at d = 32 two) tiles of O^T
          uint32_t u[2][2];  // [channels' halves][keys' halves], two keys side by side
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            u[0][h] = __byte_perm(vw[h][0][x], vw[h][1][x], 0x5410);
            u[1][h] = __byte_perm(vw[h][0][x], vw[h][1][x], 0x7632);
          }
          if constexpr (D == 32) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              b[0][2 * h] = q4_pair<0>(u[0][h], sc[h]);
              b[0][2 * h + 1] = q4_pair<1>(u[0][h], sc[h]);
              b[1][2 * h] = q4_pair<2>(u[0][h], sc[h]);
              b[1][2 * h + 1] = q4_pair<3>(u[0][h], sc[h]);
            }
          } else {
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int r = 0; r < 2; ++r) {
                b[0][2 * h + r] = q4_pair<0>(u[r][h], sc[h]);
                b[1][2 * h + r] = q4_pair<1>(u[r][h], sc[h]);
                b[2][2 * h + r] = q4_pair<2>(u[r][h], sc[h]);
                b[3][2 * h + r] = q4_pair<3>(u[r][h], sc[h]);
              }
          }
          constexpr int N = D == 32 ? 2 : 4;
#pragma unroll
          for (int v = 0; v < G; ++v) {
#pragma unroll
            for (int n = 0; n < N; ++n) q4_mma(o[v][4 * x + n], b[n], hi[v][0], hi[v][1]);
            if constexpr (!both) {
#pragma unroll
              for (int n = 0; n < N; ++n) q4_mma(o[v][4 * x + n], b[n], lo[v][0], lo[v][1]);
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

    // the warps' sums over their keys, then out or this CTA's part.  The rows
    // of O^T's tiles are D / 8 consecutive channels (at d = 32 every other one).
    if constexpr (both) {
#pragma unroll
      for (int n = 0; n < MT; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[0][n][j] += __shfl_xor_sync(0xffffffffu, o[0][n][j], 2);
    }
#pragma unroll
    for (int u = 0; u < G; ++u) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int row = 8 * u + 2 * t4 + e;
        if (row < rows) {
          float* dst = red + (warp * a.red_rows + row) * RS;
          if constexpr (D == 32) {
#pragma unroll
            for (int n = 0; n < 4; ++n) dst[8 * (g8 >> 1) + 2 * n + (g8 & 1)] = o[u][n >> 1][2 * (n & 1) + e];
          } else {
#pragma unroll
            for (int n = 0; n < MT; n += 2)
              *reinterpret_cast<float4*>(dst + g8 * (D / 8) + 2 * n) =
                  make_float4(o[u][n][e], o[u][n][2 + e], o[u][n + 1][e], o[u][n + 1][2 + e]);
          }
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
    uint16_t* out = a.out + ((long long)(g.seq.q0 + w.tile_rows * g.qt) * w.heads + g.h) * D;
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

template <int D, int TOKENS, bool CLUSTER>
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
    q4_compute<D, TOKENS, CLUSTER>(a, pool, w, c, g, smem_raw + (base - raw), full, empty, red, m, wt);
  if constexpr (CLUSTER) step_cluster_join<D, C::THREADS>(a, g, rank, red, &m->abort_flag);
}

// The kernels' shared memory, once a device.
template <int D>
cudaError_t q4_prepare() {
  static DeviceOnce once;
  return once.run([] {
    cudaError_t e = cudaSuccess;
    auto allow = [&e](const void* kernel) {
      if (e == cudaSuccess)
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kQ4BytesMost<D>);
    };
    allow(reinterpret_cast<const void*>(step_q4_kernel<D, 4, false>));
    allow(reinterpret_cast<const void*>(step_q4_kernel<D, 4, true>));
    allow(reinterpret_cast<const void*>(step_q4_kernel<D, 8, false>));
    allow(reinterpret_cast<const void*>(step_q4_kernel<D, 8, true>));
    allow(reinterpret_cast<const void*>(step_q4_kernel<D, 16, false>));
    allow(reinterpret_cast<const void*>(step_q4_kernel<D, 16, true>));
    return e;
  });
}

template <int D>
cudaError_t clusters_q4(int* n) {
  const cudaError_t e = q4_prepare<D>();
  if (e != cudaSuccess) return e;
  return clusters_at_once(step_q4_kernel<D, 16, true>, Q4Cfg<D>::THREADS, kQ4BytesMost<D>, n);
}

template <int D, int TOKENS>
cudaError_t launch_step_q4_t(const Q4Pool& pool, long long most, bool clusters, StepArgs a, int sms,
                             cudaStream_t stream) {
  using C = Q4Cfg<D>;
  a.stages = C::STAGES;
  const int bytes = a.stages * C::STAGEB + q4_red_bytes(C::WARPS, a.red_rows, D) + kQ4TailBytes + 128;
  const cudaError_t e = q4_prepare<D>();
  if (e != cudaSuccess) return e;
  if (clusters)
    return launch_after_in_clusters(kStepCluster, step_q4_kernel<D, TOKENS, true>,
                                    kStepCluster * a.w.tiles * a.p.batch * a.w.heads, C::THREADS, bytes,
                                    stream, a, pool);
  const int grid = (int)std::min<long long>((long long)C::PER_SM * sms, most);
  return launch_after(step_q4_kernel<D, TOKENS, false>, grid, C::THREADS, bytes, stream, a, pool);
}
template <int D>
cudaError_t launch_step_q4_d(const Q4Pool& pool, long long most, bool clusters, const StepArgs& a, int sms,
                             cudaStream_t stream) {
  // red_rows: the most new tokens that a tile can hold
  if (a.red_rows <= 4) return launch_step_q4_t<D, 4>(pool, most, clusters, a, sms, stream);
  if (a.red_rows <= 8) return launch_step_q4_t<D, 8>(pool, most, clusters, a, sms, stream);
  return launch_step_q4_t<D, 16>(pool, most, clusters, a, sms, stream);
}

template <int D>
cudaError_t launch_append_q4_d(const Q4Pool& pool, AppendArgs a, int sms, cudaStream_t stream) {
  a.check_ctas = q4_check_ctas(a.p);
  const int step = q4_head_step<D, kQ4AppendIter>(a.p.rows, a.heads, sms);
  const int grid = (int)(a.check_ctas + q4_blocks<D, kQ4AppendIter>(a.p.rows, a.heads, step));
  return launch_after(append_q4_kernel<D>, grid, kQ4Threads, 0, stream, a, pool, step);
}

template <int D>
cudaError_t launch_read_q4_d(const Q4Pool& pool, ReadArgs a, int sms, cudaStream_t stream) {
  a.check_ctas = q4_check_ctas(a.p);
  const int step = q4_head_step<D, kQ4ReadIter>(a.p.rows, a.heads, sms);
  const int grid = (int)(a.check_ctas + q4_blocks<D, kQ4ReadIter>(a.p.rows, a.heads, step));
  return launch_after(read_q4_kernel<D>, grid, kQ4Threads, 0, stream, a, pool, step);
}

}  // namespace

bool q4_rows_fit(const PagedView& p, int heads, int d) {
  // the append's CTAs, which are more than the reading's
  const long long blocks = d == 32   ? q4_blocks<32, kQ4AppendIter>(p.rows, heads, 1)
                           : d == 64 ? q4_blocks<64, kQ4AppendIter>(p.rows, heads, 1)
                                     : q4_blocks<128, kQ4AppendIter>(p.rows, heads, 1);
  static_assert(kQ4AppendIter <= kQ4ReadIter, "more CTAs");
  return q4_check_ctas(p) + blocks <= 0x7fffffffLL;
}

cudaError_t launch_append_q4(const Q4Pool& pool, const AppendArgs& a, int sms, cudaStream_t stream) {
  switch (a.d) {
    case 32: return launch_append_q4_d<32>(pool, a, sms, stream);
    case 64: return launch_append_q4_d<64>(pool, a, sms, stream);
    default: return launch_append_q4_d<128>(pool, a, sms, stream);
  }
}

cudaError_t launch_read_q4(const Q4Pool& pool, const ReadArgs& a, int sms, cudaStream_t stream) {
  switch (a.d) {
    case 32: return launch_read_q4_d<32>(pool, a, sms, stream);
    case 64: return launch_read_q4_d<64>(pool, a, sms, stream);
    default: return launch_read_q4_d<128>(pool, a, sms, stream);
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
