// Attention over kept key blocks with changed scores: capped by a tanh, lowered with the
// distance of the positions, masked by document and by order (sm_100a, tcgen05).
//
// Mathematics, per query t of a head and key u of a kept block (log2 domain):
//   z = C tanh(scale s / c)          C = c log2 e, or scale log2 e * s without a cap
//   z = z - slope log2 e |pos_t - pos_u|
//   z = -inf  unless doc_t = doc_u >= 0 and order_u <= order_t
//   m = max z,  l = sum 2^(z - m),  out = sum 2^(z - m) v / l,  lse = ln 2 (m + log2 l)
// with the running m and l of an online softmax in fp32, and products of bf16 operands
// accumulated in fp32 by the tensor cores.  P is rounded to bf16 for the second product; l
// sums the unrounded values.
//
// Work split.  One CTA per (batch, head, query block of 128) row; two CTAs share an SM.  A
// CTA first walks its list of kept blocks against the blocks' summaries (smallest and
// largest document and order, one int4 per key block, written by summary_kernel) and keeps
// in shared memory the blocks that some query of the row sees, with a class for each softmax
// warp: whole (its 32 queries see every key), none, or mixed.  Blocks that nobody sees cost
// no load and no product; only mixed tiles test element by element, and a warp that sees
// nothing of a tile stores zero weights.  When the rows are few, `splits` CTAs share a row:
// each takes a contiguous part of its tiles and writes its unnormalised sums, and
// join_kernel weighs them together.
//
// Warp roles are those of k_attn.cu (192 threads): warps 0-3 softmax, one query row per
// thread; warp 4 the TMA producer; warp 5 the tensor-core issuer.  Tensor memory: S columns
// [0,128), P [128,192), O [192,256).
//
// Masked values.  P of a masked pair is exactly 0, but 0 times an infinite or NaN value is
// NaN inside the matrix product.  A masked call therefore looks at its finished rows: if one
// that saw a key is not finite, the CTA walks its tiles a second time, and there the softmax
// warps look at the values of every tile that is not whole for all of them; those that are
// not finite are added by hand to the rows that see their token, and replaced by 0 in shared
// memory before the product.  Finite inputs pay 64 tests per row for this.
//
// What bounds it: as in k_attn.cu the softmax warps, two a scheduler, whose dependent chains do
// not hide one another; the exponentials alone take 1024 of about 1870 clocks per tile and SM.
// Measured on one B200, 16 heads x 10992 tokens, every block: 755 us plain (653 TFLOP/s), 908
// with a bias by view, 960 by token, 922 capped at 50, 2100 capped at 10 (scores beyond the
// polynomials), 1470 capped at 50 with a bias by view, 458 causal over views, 398 causal; 43968
// tokens causal over views and capped 7.1-7.2 ms (570 TFLOP/s of visible pairs).
#include <algorithm>
#include <cfloat>
#include <climits>
#include <cmath>

#include "k_attn.cuh"
#include "k_masked.cuh"

namespace ress {
namespace {

constexpr int kThreads = 192;
constexpr int kWarps = kThreads / 32;
constexpr int kProducerWarp = 4;
constexpr int kMmaWarp = 5;
constexpr float kRescaleLog2 = 8.0f;  // O and l are rescaled when the max grows by more
constexpr int kKStages = 3;
constexpr int kVStages = 2;
constexpr int kTile = 128 * 64 * 2;  // bytes of one 128 x 64 bf16 tile
constexpr int kOffQ = 0;
constexpr int kOffK = kTile;
constexpr int kOffV = kOffK + kKStages * kTile;
constexpr int kOffList = kOffV + kVStages * kTile;   // uint16 per kept block: its index
constexpr int kOffClass = kOffList + 2 * kMaxBlocks;  // uint8: two bits per softmax warp
constexpr int kOffMeta = kOffClass + kMaxBlocks;      // a mixed tile's documents and orders
constexpr int kOffPos = kOffMeta + 2 * 128 * 4;       // per softmax warp: the tile's positions
constexpr int kOffBar = kOffPos + 4 * 128 * 4;
constexpr int kSmemBytes = kOffBar + 384 + 1024;
static_assert(2 * (kSmemBytes + 1024) <= 228 * 1024, "two CTAs per SM");
constexpr uint32_t kTmemCols = 256;
constexpr uint32_t kColS = 0, kColP = 128, kColO = 192;
constexpr int kUneven = INT_MIN;  // step of a block whose positions do not run evenly
constexpr uint32_t kWhole = 0, kMixed = 1, kNone = 2;  // what a warp sees of a block

struct Bars {
  uint64_t q_full;
  uint64_t k_full[kKStages];
  uint64_t k_empty[kKStages];
  uint64_t v_full[kVStages];
  uint64_t v_empty[kVStages];
  uint64_t s_full;
  uint64_t s_free;
  uint64_t p_full;
  uint64_t o_done;
  uint64_t o_half;
  uint64_t drain;
  uint64_t meet;  // the softmax warps meet: around a mixed tile's arrays and a tile's values
  uint32_t tmem_base;
  // the row, for the softmax loop: kept here because its registers are full
  int b, bh, qi, active, skip, tiles, entries;
  int abort;
  int o_init;           // O was started by hand: the first product adds to it
  int count[kWarps];    // filter: visible blocks of each warp's entries
  int qsum[4][5];       // filter: each softmax warp's query summary
  uint32_t vflag[4];    // rows of V (32 per word) that hold a value that is not finite
};
static_assert(sizeof(Bars) <= 384, "barriers fit their shared-memory slot");

RESS_DEV void fence_async_shared() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// s <- tanh(s in) of a row's 128 scores, by the polynomial.
template <int N>
RESS_DEV void cap_small(uint32_t (&sv)[128], float in) {
  const uint64_t in2 = f2(in, in);
#pragma unroll
  for (int c = 0; c < 128; c += 2) {
    const uint64_t y = fmul2(f2(__uint_as_float(sv[c]), __uint_as_float(sv[c + 1])), in2);
    const uint64_t t = fmul2(y, y);
    uint64_t a = f2(tanh_fit<N>(N), tanh_fit<N>(N));
#pragma unroll
    for (int k = N - 1; k >= 0; --k) a = ffma2(a, t, f2(tanh_fit<N>(k), tanh_fit<N>(k)));
    const uint64_t u = fmul2(a, y);
    sv[c] = __float_as_uint(f2lo(u));
    sv[c + 1] = __float_as_uint(f2hi(u));
  }
}
// Any score, as tanh_any: 1 - 2 / (1 + e^2y) from |y| = 1/2 on, the polynomial below, so that
// small scores beside large ones keep a relative error (2^-21 of each score's own).
RESS_DEV void cap_any(uint32_t (&sv)[128], float in) {
  const float in2 = 2.0f * kLog2e * in, half = 0.5f / in;
  const uint64_t ins = f2(in, in);
#pragma unroll
  for (int c = 0; c < 128; c += 2) {
    const float s[2] = {__uint_as_float(sv[c]), __uint_as_float(sv[c + 1])};
    const uint64_t y = fmul2(f2(s[0], s[1]), ins);
    const uint64_t t = fmul2(y, y);
    uint64_t a = f2(tanh_fit<4>(4), tanh_fit<4>(4));
#pragma unroll
    for (int k = 3; k >= 0; --k) a = ffma2(a, t, f2(tanh_fit<4>(k), tanh_fit<4>(k)));
    const uint64_t u = fmul2(a, y);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float r = rcp_approx(1.0f + ex2_approx(s[i] * in2));
      sv[c + i] = __float_as_uint(fabsf(s[i]) < half ? (i ? f2hi(u) : f2lo(u)) : fmaf(-2.0f, r, 1.0f));
    }
  }
}

// Programmatic dependent launch: a kernel's CTAs may start while the kernel before it still
// runs, once all of that one's CTAs have called launch_dependents (or ended), and wait for its
// results where they need them.  Without the launch attribute both do nothing.  Such results are
// never read as constants (__ldg, const __restrict__): they are still being written when the
// reader starts, and the read-only path may serve a load from before the wait.
RESS_DEV void launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
RESS_DEV void wait_prerequisites() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

struct Params {
  const int32_t *kv_idx, *kv_cnt, *order;
  const int32_t *q_pos, *k_pos, *q_doc, *k_doc, *q_order, *k_order;
  const float *slopes;
  // [2][B][nk]: smallest and largest document, smallest and largest order of each key block;
  // and its smallest, largest and first position with the step from token to token
  const int4 *blocks;
  __nv_bfloat16 *out;
  float *lse;
  float *part_o;    // [items][splits][128][64]
  float2 *part_ml;  // [items][splits][128]
  int32_t *dev_err;
  int B, H, N, Nq, nq, nk;
  int splits;
  float scale_log2;         // without a cap
  float cap_log2, cap_in;   // c log2 e; scale / c
  float cap_half;           // scores up to this stay within |y| = 1/2
  float cap_a, cap_k[4];    // and up to this (|y| = 3/8, |z| = 32) the cap is s cap_k(s^2), log2 domain
};

// KB tokens per key block; CAP, BIAS: the score changes compiled in.
template <int KB, bool CAP, bool BIAS>
__global__ void __launch_bounds__(kThreads, 2)
    masked_attn_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                       const __grid_constant__ CUtensorMap tmV, const __grid_constant__ Params p) {
  extern __shared__ unsigned char smem_raw[];
  // an offset, not a rounded pointer: the compiler still sees shared memory (32-bit addresses)
  unsigned char *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  Bars *bar = reinterpret_cast<Bars *>(smem + kOffBar);
  uint16_t *list = reinterpret_cast<uint16_t *>(smem + kOffList);
  uint8_t *classes = smem + kOffClass;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  // rows of a head from its last query block to its first: under an order mask the long
  // rows start first, and a head's keys stay in L2 while its rows run
  launch_dependents();
  if (p.order) wait_prerequisites();  // (an order of our own is written by the kernel before)
  const int x = blockIdx.x;
  const int item32 = p.order ? p.order[x] : x / p.nq * p.nq + (p.nq - 1 - x % p.nq);
  if (p.order && (item32 < 0 || item32 >= (int)gridDim.x)) {  // not a permutation
    if (tid == 0) report_error(p.dev_err, RESS_ERR_DEVICE_BOUNDS);
    return;
  }
  const int bh = item32 / p.nq, qi = item32 - bh * p.nq, b = bh / p.H;
  const long long item = item32;
  const bool masked = p.q_doc != nullptr || p.q_order != nullptr;

  // softmax warps that hold a query (the others stay out: their rows of S, P and O are
  // never read)
  const int active = min(4, (p.Nq - qi * 128 + 31) >> 5);

  if (tid == kProducerWarp * 32) {
    // the queries load while the row's blocks are looked up
    mbar_init(&bar->q_full, 1);
    fence_mbar_init();
    tma_prefetch_desc(&tmQ);
    mbar_arrive_expect_tx(&bar->q_full, kTile);
    tma_load_3d(smem + kOffQ, &tmQ, &bar->q_full, 0, qi * 128, bh);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  if (tid == 0) {
    for (int s = 0; s < kKStages; ++s) {
      mbar_init(&bar->k_full[s], 1);
      mbar_init(&bar->k_empty[s], 1);
    }
    for (int s = 0; s < kVStages; ++s) {
      mbar_init(&bar->v_full[s], 1);
      mbar_init(&bar->v_empty[s], 1);
    }
    mbar_init(&bar->s_full, 1);
    mbar_init(&bar->s_free, active);
    mbar_init(&bar->p_full, active);
    mbar_init(&bar->o_done, 1);
    mbar_init(&bar->o_half, 1);
    mbar_init(&bar->drain, 1);
    mbar_init(&bar->meet, active);
    bar->abort = 0;
    bar->o_init = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&bar->tmem_base, kTmemCols);
    tmem_relinquish();
  }

  // ---------------------------------------------------------------- the row's blocks
  // the loads of this thread's first entry go out before the queries' arrays are looked at
  wait_prerequisites();  // the summaries
  const int cnt = p.kv_cnt ? p.kv_cnt[item] : p.nk;
  const int32_t *kvrow = p.kv_idx ? p.kv_idx + item * p.nk : nullptr;
  const int kb0 = kvrow ? (tid < p.nk ? kvrow[tid] : -1) : tid;  // (past cnt: anything)
  int4 sum0 = make_int4(0, 0, 0, 0);
  if (masked && kb0 >= 0 && kb0 < p.nk) sum0 = p.blocks[(long long)b * p.nk + kb0];
  const int t = qi * 128 + tid;  // query token of a softmax thread
  if (warp < 4) {
    int row_doc = 0, row_order = 0;
    const bool there = t < p.Nq;
    if (p.q_doc) row_doc = there ? p.q_doc[(long long)b * p.Nq + t] : -1;
    if (p.q_order) row_order = there ? p.q_order[(long long)b * p.Nq + t] : 0;
    // over the rows that may see something: documents, orders, and whether some see nothing
    const bool live = there && row_doc >= 0;
    int v[5] = {live ? row_doc : INT_MAX, live ? row_doc : INT_MIN, live ? row_order : INT_MAX,
                live ? row_order : INT_MIN, there && row_doc < 0};
    v[0] = __reduce_min_sync(0xffffffffu, v[0]);
    v[1] = __reduce_max_sync(0xffffffffu, v[1]);
    v[2] = __reduce_min_sync(0xffffffffu, v[2]);
    v[3] = __reduce_max_sync(0xffffffffu, v[3]);
    v[4] = __reduce_or_sync(0xffffffffu, v[4]);
    if (lane == 0)
      for (int i = 0; i < 5; ++i) bar->qsum[warp][i] = v[i];
  }
  __syncthreads();
  const bool ragged = p.N % KB != 0;
  bool bad = cnt < 0 || cnt > p.nk;
  int kept = 0;
  if (!bad) {
    for (int j0 = 0; j0 < cnt; j0 += kThreads) {
      const int j = j0 + tid;
      int kb = -1;
      bool see = false;
      uint32_t cls = 0;
      if (j < cnt) {
        kb = j0 == 0 ? kb0 : (kvrow ? kvrow[j] : j);
        if (kb < 0 || kb >= p.nk) {
          bad = true;
        } else {
          int4 sum = sum0;
          if (masked && j0 > 0) sum = p.blocks[(long long)b * p.nk + kb];
          const bool cut = ragged && kb == p.nk - 1;
          for (int w = 0; w < active; ++w) {
            bool some = true, whole = !cut;
            const int *q = bar->qsum[w];
            if (p.q_doc) {
              some = q[1] >= 0 && sum.y >= 0 && max(sum.x, 0) <= q[1] && sum.y >= q[0];
              whole = whole && !q[4] && q[0] == q[1] && sum.x == sum.y && sum.x == q[0];
            }
            if (p.q_order) {
              some = some && sum.z <= q[3];
              whole = whole && sum.w <= q[2];
            }
            see |= some;
            cls |= (some ? (whole ? kWhole : kMixed) : kNone) << (2 * w);
          }
        }
      }
      const uint32_t seen = __ballot_sync(0xffffffffu, see);
      if (lane == 0) bar->count[warp] = __popc(seen);
      __syncthreads();
      int at = kept;
      for (int w = 0; w < kWarps; ++w) {
        const int n = bar->count[w];
        if (w < warp) at += n;
        kept += n;
      }
      if (see) {
        at += __popc(seen & ((1u << lane) - 1));
        list[at] = (uint16_t)kb;
        classes[at] = (uint8_t)cls;
      }
      __syncthreads();
    }
  }
  tc_fence_before();
  const int any_bad = __syncthreads_or(bad);
  tc_fence_after();
  const uint32_t tmem = bar->tmem_base;
  volatile int *abort = &bar->abort;
  // this CTA's tiles of the row
  const int all_tiles = KB == 128 ? kept : (kept + 1) >> 1;
  const int first = (int)((long long)all_tiles * blockIdx.y / p.splits);
  const int tiles = any_bad ? 0 : (int)((long long)all_tiles * (blockIdx.y + 1) / p.splits) - first;
  if (any_bad && tid == 0) report_error(p.dev_err, RESS_ERR_DEVICE_BOUNDS);

  if (tiles > 0) {
    const int entries = KB == 128 ? tiles : min(2 * tiles, kept - 2 * first);
    const int skip = KB == 128 ? first : 2 * first;
    const uint16_t *mine = list + skip;
    if (tid == 0) {
      bar->b = b;
      bar->bh = bh;
      bar->qi = qi;
      bar->active = active;
      bar->skip = skip;
      bar->tiles = tiles;
      bar->entries = entries;
    }
    __syncthreads();
    // A second pass over the tiles follows only where hidden values that are not finite have
    // to be kept out of the products; J counts tiles over both, for the barriers' phases.
    int meets = 0;
    for (int pass = 0;; ++pass) {
      const int J0 = pass * tiles;
      bool again = false;
      float m_run = kNoMax, l_run = 0.f;
      bool ok = true;
      if (warp == kProducerWarp) {
        // ---------------------------------------------------------- TMA producer
        if (lane == 0) {
          // one 128-row box, or two 64-row boxes (row N, past the last token, reads as zero
          // where the row has no second block)
          auto load_tile = [&](const CUtensorMap *tm, unsigned char *dst, uint64_t *full, int j) {
            mbar_arrive_expect_tx(full, kTile);
            if constexpr (KB == 128) {
              tma_load_3d(dst, tm, full, 0, mine[j] * 128, bh);
            } else {
              const int r1 = 2 * j + 1 < entries ? mine[2 * j + 1] * 64 : p.N;
              tma_load_3d(dst, tm, full, 0, mine[2 * j] * 64, bh);
              tma_load_3d(dst + kTile / 2, tm, full, 0, r1, bh);
            }
          };
          // tile j waits for its slot's last user, tile J - stages
          auto load_k = [&](int j) {
            const int J = J0 + j, s = J % kKStages;
            if (J >= kKStages && !mbar_wait(&bar->k_empty[s], (J / kKStages - 1) & 1, abort)) return false;
            load_tile(&tmK, smem + kOffK + s * kTile, &bar->k_full[s], j);
            return true;
          };
          auto load_v = [&](int j) {
            const int J = J0 + j, s = J % kVStages;
            if (J >= kVStages && !mbar_wait(&bar->v_empty[s], (J / kVStages - 1) & 1, abort)) return false;
            load_tile(&tmV, smem + kOffV + s * kTile, &bar->v_full[s], j);
            return true;
          };
          int nk = 0, nv = 0;
          while (nk < min(tiles, kKStages) && load_k(nk)) ++nk;
          while (nv < min(tiles, kVStages) && load_v(nv)) ++nv;
          for (int j = 0; j < tiles; ++j) {
            if (j + kKStages < tiles) {
              if (!load_k(j + kKStages)) break;
              nk = j + kKStages + 1;
            }
            if (j + kVStages < tiles) {
              if (!load_v(j + kVStages)) break;
              nv = j + kVStages + 1;
            }
          }
          if (*abort == 0 && (nk < tiles || nv < tiles)) {
            report_error(p.dev_err, RESS_ERR_DEVICE_TIMEOUT);
            *abort = 1;
          }
          // never leave the CTA with copies in flight
          for (int j = max(0, nk - kKStages); j < nk; ++j)
            mbar_wait(&bar->k_full[(J0 + j) % kKStages], ((J0 + j) / kKStages) & 1, nullptr);
          for (int j = max(0, nv - kVStages); j < nv; ++j)
            mbar_wait(&bar->v_full[(J0 + j) % kVStages], ((J0 + j) / kVStages) & 1, nullptr);
        }
      } else if (warp == kMmaWarp) {
        // ---------------------------------------------------- tensor-core issuer
        if (lane == 0) {
          const uint32_t sQ = smem_u32(smem + kOffQ);
          const uint32_t sK = smem_u32(smem + kOffK);
          const uint32_t sV = smem_u32(smem + kOffV);
          volatile int *o_init = &bar->o_init;
          ok = mbar_wait(&bar->q_full, 0, abort);
          tc_fence_after();
          const uint64_t dq = smem_desc(sQ);
          for (int j = 0; ok && j <= tiles; ++j) {
            const int J = J0 + j;
            if (j < tiles) {
              const int s = J % kKStages;
              ok = mbar_wait(&bar->k_full[s], (J / kKStages) & 1, abort);
              if (ok && J > 0) ok = mbar_wait(&bar->s_free, (J - 1) & 1, abort);
              if (!ok) break;
              tc_fence_after();
              const uint64_t dk = smem_desc(sK + s * kTile);
#pragma unroll
              for (int k = 0; k < 4; ++k) mma_ss(tmem + kColS, dq + 2 * k, dk + 2 * k, kIdescS, k > 0);
              mma_commit(&bar->s_full);
              mma_commit(&bar->k_empty[s]);
            }
            if (j > 0) {
              const int Jp = J - 1, sp = Jp % kVStages;
              ok = mbar_wait(&bar->p_full, Jp & 1, abort);
              if (ok) ok = mbar_wait(&bar->v_full[sp], (Jp / kVStages) & 1, abort);
              if (!ok) break;
              tc_fence_after();
              const uint64_t dv = smem_desc(sV + sp * kTile);
              const bool add = j > 1 || *o_init != 0;
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                mma_ts(tmem + kColO, tmem + kColP + 8 * k, dv + 128 * k, kIdescPV, (add || k > 0));
                if (k == 3) mma_commit(&bar->o_half);
              }
              mma_commit(&bar->o_done);
              mma_commit(&bar->v_empty[sp]);
            }
          }
          if (!ok) {
            report_error(p.dev_err, RESS_ERR_DEVICE_TIMEOUT);
            *abort = 1;
          }
          // drain: every MMA issued above has finished before the CTA tears down
          mma_commit(&bar->drain);
          mbar_wait(&bar->drain, pass & 1, nullptr);
        }
      } else if (warp < active) {
        // ----------------------------------------------------------- softmax
        const volatile Bars *vb = bar;
        const uint32_t trow = vb->tmem_base + ((uint32_t)(warp * 32) << 16);
        int *m_doc = reinterpret_cast<int *>(smem + kOffMeta), *m_order = m_doc + 128;
        float *m_pos = reinterpret_cast<float *>(smem + kOffPos) + warp * 128;
        int q_pos = 0, q_lo = 0, q_hi = 0;  // this query's position, and the range of the warp's
        float slope = 0.f;
        if constexpr (BIAS) {
          q_pos = p.q_pos[(long long)vb->b * p.Nq + min(vb->qi * 128 + tid, p.Nq - 1)];
          q_lo = __reduce_min_sync(0xffffffffu, q_pos);
          q_hi = __reduce_max_sync(0xffffffffu, q_pos);
          slope = -p.slopes[vb->bh % p.H] * kLog2e;
        }
        // key of column c of tile j, or -1
        auto key_of = [&](int j, int c) {
          const volatile uint16_t *own = list + vb->skip;
          int u;
          if constexpr (KB == 128) {
            u = own[j] * 128 + c;
          } else {
            if (c >= 64 && 2 * j + 1 >= vb->entries) return -1;
            u = own[2 * j + (c >> 6)] * 64 + (c & 63);
          }
          return u < p.N ? u : -1;
        };
        // A wait that gives up does not leave the tile: the lanes stay together, later waits
        // return at once (abort), and the loop ends after a vote.
        auto wait = [&](uint64_t *which, uint32_t parity) {
          if (!mbar_wait(which, parity, abort)) {
            ok = false;
            *abort = 1;
          }
        };
        auto meet = [&]() {  // the softmax warps meet
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar->meet);
          wait(&bar->meet, meets & 1);
          ++meets;
        };
        for (int j = 0; j < vb->tiles; ++j) {
          const int J = (pass ? vb->tiles : 0) + j;
          // the warps' classes of this tile: of its block, or of its two
          const volatile uint8_t *own = classes + vb->skip + (KB == 128 ? j : 2 * j);
          uint32_t cls = own[0];
          if constexpr (KB == 64) {
            const uint32_t c1 = 2 * j + 1 < vb->entries ? own[1] : 0xAAu;
            const uint32_t differ = ((cls ^ c1) | ((cls ^ c1) >> 1)) & 0x55u;
            cls = (cls & ~(3u * differ)) | differ;
          }
          cls &= (1u << (2 * vb->active)) - 1;
          const uint32_t code = (cls >> (2 * warp)) & 3;
          if (cls & ~(cls >> 1) & 0x55u) {  // mixed for some warp
            meet();  // the last mixed tile's arrays have been read
            for (int c = tid; c < 128; c += 32 * vb->active) {
              const int u = key_of(j, c);
              const long long at = (long long)vb->b * p.N + u;
              m_doc[c] = u < 0 ? -1 : (p.k_doc ? max(__ldg(p.k_doc + at), -1) : 0);
              m_order[c] = u < 0 || !p.k_order ? 0 : __ldg(p.k_order + at);
            }
            meet();
          }
          // The bias of column c of half i, where the keys lie on one side of the warp's
          // queries: shift[i] + step[i] (c mod 64 - end) if positions run evenly in each half
          // (the usual case: tokens, or all of one view), else shift[i] + m_pos[c].  end is
          // the column of a half's key nearest to the queries, 0 or 63; m_pos is measured from
          // the warp's query nearest to the keys: both terms have the distance's sign, and
          // neither is larger, so that nothing cancels however far the tile reaches and
          // wherever the block's other queries are.  On both sides, from the middle of all
          // of the positions: differences from it are exact up to the documented 2^24.
          float shift[2] = {0.f, 0.f}, step[2] = {0.f, 0.f};
          int side = 0;  // +1: every key at or before every query, -1: at or after, 0: mixed
          bool even = true, last = false;  // last: end = 63
          float row_pos = 0.f;
          if constexpr (BIAS) {
            // (summaries are 16 bytes a block: eight of them to a line of L1)
            const volatile uint16_t *own = list + vb->skip + (KB == 128 ? j : 2 * j);
            const int4 *sum = p.blocks + (long long)(p.B + vb->b) * p.nk;
            const int4 p0 = sum[own[0]];  // smallest, largest, first, step
            const int4 p1 = KB == 64 && 2 * j + 1 < vb->entries ? sum[own[1]] : p0;
            const int lo = min(p0.x, p1.x), hi = max(p0.y, p1.y);
            side = hi <= q_lo ? 1 : (lo >= q_hi ? -1 : 0);
            even = side != 0 && p0.w != kUneven && p1.w != kUneven && (p0.w >= 0) == (p1.w >= 0);
            last = side > 0 ? max(p0.w, p1.w) > 0 : min(p0.w, p1.w) < 0;
            const float f = side == 0 ? 1.0f : (side > 0 ? -slope : slope);
            if (even) {
              step[0] = f * (float)p0.w;
              step[1] = f * (float)p1.w;
              const int end = last ? 63 : 0;
              shift[0] = f * (float)((long long)p0.z - q_pos + (long long)end * p0.w);
              shift[1] = f * (float)((long long)p1.z - q_pos + (long long)((KB == 64 ? 0 : 64) + end) * p1.w);
            } else {
              const int ref = side > 0 ? q_lo : (side < 0 ? q_hi : (int)(((long long)min(q_lo, lo) + max(q_hi, hi)) >> 1));
              row_pos = (float)((long long)q_pos - ref);
              shift[0] = shift[1] = side == 0 ? 0.f : -f * row_pos;
              __syncwarp();  // the last tile's have been read
              for (int c = lane; c < 128; c += 32) {
                const int u = max(key_of(j, c), 0);  // (a column without a key is masked)
                m_pos[c] = (float)((long long)__ldg(p.k_pos + (long long)vb->b * p.N + u) - ref) * f;
              }
              __syncwarp();
            }
          }
          wait(&bar->s_full, J & 1);
          tc_fence_after();
          uint32_t sv[128];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            tmem_ld32(trow + kColS + 32 * i, *reinterpret_cast<uint32_t(*)[32]>(&sv[32 * i]));
          tmem_wait_ld();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar->s_free);
          bool rescale = false;
          float alpha = 1.0f, m_use = m_run;
          uint32_t pk[64];
          // P and its sum from the exponents of column pairs
          auto weights = [&](auto z_of) {
            constexpr int kChains = CAP ? 2 : 4;  // sums; the cap leaves fewer registers
            uint64_t acc[kChains] = {};
#pragma unroll
            for (int c = 0; c < 64; ++c) {
              const uint64_t z = z_of(c);
              const uint64_t e = f2(ex2_approx(f2lo(z)), ex2_approx(f2hi(z)));
              acc[c % kChains] = fadd2(acc[c % kChains], e);
              pk[c] = pack_bf16x2(f2lo(e), f2hi(e));
              if (c == 31) {
                // keys 0..63 of P: free once the first half of the previous product is done
                if (j > 0) wait(&bar->o_half, (J - 1) & 1);
                tmem_st32(trow + kColP, *reinterpret_cast<uint32_t(*)[32]>(&pk[0]));
              }
            }
            uint64_t a = fadd2(acc[0], acc[1]);
            if (kChains == 4) a = fadd2(a, fadd2(acc[kChains - 2], acc[kChains - 1]));
            alpha = rescale ? ex2_approx(m_run - m_use) : 1.0f;
            l_run = l_run * alpha + (f2lo(a) + f2hi(a));
            m_run = m_use;
          };
          auto raise = [&](float m_new) {
            rescale = m_new > m_run + kRescaleLog2;
            m_use = rescale ? m_new : m_run;
          };
          float big = 0.f;  // largest |score|, for the cap of a whole tile
          bool fused = false;
          if constexpr (CAP) {
            float mc[2] = {0.f, 0.f};
#pragma unroll
            for (int c = 0; c < 128; c += 4) {
#pragma unroll
              for (int q = 0; q < 2; ++q)
                mc[q] = fmax3(mc[q], fabsf(__uint_as_float(sv[c + 2 * q])), fabsf(__uint_as_float(sv[c + 2 * q + 1])));
            }
            // (a mixed tile's may be a hidden key's, which must not choose the visible ones'
            // arithmetic: such a tile takes the form for any score)
            big = code == kWhole ? fmaxf(mc[0], mc[1]) : INFINITY;
            fused = !BIAS && __all_sync(0xffffffffu, big <= p.cap_a);
          }
          if (code == kNone) {
#pragma unroll
            for (int c = 0; c < 64; ++c) pk[c] = 0u;
            if (j > 0) wait(&bar->o_half, (J - 1) & 1);
            tmem_st32(trow + kColP, *reinterpret_cast<uint32_t(*)[32]>(&pk[0]));
          } else if (CAP && !BIAS && fused) {
            // the cap inside the exponent, s P(s^2) with the scales in its coefficients; the
            // cap of the largest |s| bounds the row's scores
            const float y = big * big;
            raise(fmaxf(m_run, big * fmaf(fmaf(fmaf(p.cap_k[3], y, p.cap_k[2]), y, p.cap_k[1]), y, p.cap_k[0])));
            const uint64_t k0 = f2(p.cap_k[0], p.cap_k[0]), k1 = f2(p.cap_k[1], p.cap_k[1]);
            const uint64_t k2 = f2(p.cap_k[2], p.cap_k[2]), k3 = f2(p.cap_k[3], p.cap_k[3]);
            const uint64_t nm = f2(-m_use, -m_use);
            weights([&](int c) {
              const uint64_t s2 = f2(__uint_as_float(sv[2 * c]), __uint_as_float(sv[2 * c + 1]));
              const uint64_t t = fmul2(s2, s2);
              return ffma2(ffma2(ffma2(ffma2(k3, t, k2), t, k1), t, k0), s2, nm);
            });
          } else {
            // z = sv * sc + shift from here on
            float sc = p.scale_log2;
            if constexpr (CAP) {
              if (__all_sync(0xffffffffu, big <= p.cap_half))
                cap_small<4>(sv, p.cap_in);
              else if (__all_sync(0xffffffffu, big <= 2.0f * p.cap_half))
                cap_small<6>(sv, p.cap_in);
              else
                cap_any(sv, p.cap_in);
              sc = p.cap_log2;
            }
            if constexpr (BIAS) {
              const uint64_t sc2 = f2(sc, sc);
              if (!even || step[0] != 0.f || step[1] != 0.f) {
                if (even) {
                  // from the near end outwards, so that the running sum's roundings are of its
                  // own size (a product with the column's number each: 1050 against 944 us)
                  const auto ramp = [&](bool back) {  // (known when this is unrolled)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                      const float t = back ? -step[i] : step[i];
                      const uint64_t st = f2(8.0f * t, 8.0f * t);
                      uint64_t run[4];
#pragma unroll
                      for (int q = 0; q < 4; ++q)
                        run[q] = back ? f2((2 * q + 1) * t, 2 * q * t) : f2(2 * q * t, (2 * q + 1) * t);
#pragma unroll
                      for (int c = 0; c < 64; c += 2) {
                        uint32_t *s = &sv[64 * i + (back ? 62 - c : c)];
                        const int q = (c >> 1) & 3;
                        const uint64_t z = ffma2(f2(__uint_as_float(s[0]), __uint_as_float(s[1])), sc2, run[q]);
                        run[q] = fadd2(run[q], st);
                        s[0] = (uint32_t)z;
                        s[1] = (uint32_t)(z >> 32);
                      }
                    }
                  };
                  last ? ramp(true) : ramp(false);
                } else if (side != 0) {
#pragma unroll
                  for (int c = 0; c < 128; c += 4) {
                    const ulonglong2 kp = *reinterpret_cast<const ulonglong2 *>(m_pos + c);
                    const uint64_t z0 = ffma2(f2(__uint_as_float(sv[c]), __uint_as_float(sv[c + 1])), sc2, kp.x);
                    const uint64_t z1 = ffma2(f2(__uint_as_float(sv[c + 2]), __uint_as_float(sv[c + 3])), sc2, kp.y);
                    sv[c] = (uint32_t)z0;
                    sv[c + 1] = (uint32_t)(z0 >> 32);
                    sv[c + 2] = (uint32_t)z1;
                    sv[c + 3] = (uint32_t)(z1 >> 32);
                  }
                } else {
#pragma unroll
                  for (int c = 0; c < 128; c += 4) {
                    const float4 kp = *reinterpret_cast<const float4 *>(m_pos + c);
                    const float d[4] = {fabsf(row_pos - kp.x), fabsf(row_pos - kp.y), fabsf(row_pos - kp.z),
                                        fabsf(row_pos - kp.w)};
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                      sv[c + i] = __float_as_uint(fmaf(slope, d[i], __uint_as_float(sv[c + i]) * sc));
                  }
                }
                sc = 1.0f;
              }
            }
            if (code == kMixed) {
              const int t = vb->qi * 128 + tid;
              {
                int row_doc = 0;  // (a column without a key has document -1)
                if (p.q_doc) row_doc = t < p.Nq ? __ldg(p.q_doc + (long long)vb->b * p.Nq + t) : -1;
                if (row_doc < 0) row_doc = -2;  // equal to no key's document
#pragma unroll
                for (int c = 0; c < 128; c += 4) {
                  const int4 kd = *reinterpret_cast<const int4 *>(m_doc + c);
                  if (kd.x != row_doc) sv[c] = __float_as_uint(-INFINITY);
                  if (kd.y != row_doc) sv[c + 1] = __float_as_uint(-INFINITY);
                  if (kd.z != row_doc) sv[c + 2] = __float_as_uint(-INFINITY);
                  if (kd.w != row_doc) sv[c + 3] = __float_as_uint(-INFINITY);
                }
              }
              if (p.q_order) {
                const int row_order = t < p.Nq ? __ldg(p.q_order + (long long)vb->b * p.Nq + t) : 0;
#pragma unroll
                for (int c = 0; c < 128; c += 4) {
                  const int4 ko = *reinterpret_cast<const int4 *>(m_order + c);
                  if (ko.x > row_order) sv[c] = __float_as_uint(-INFINITY);
                  if (ko.y > row_order) sv[c + 1] = __float_as_uint(-INFINITY);
                  if (ko.z > row_order) sv[c + 2] = __float_as_uint(-INFINITY);
                  if (ko.w > row_order) sv[c + 3] = __float_as_uint(-INFINITY);
                }
              }
            }
            float mh[2];  // maxima of the halves
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              float mc[2] = {-INFINITY, -INFINITY};
#pragma unroll
              for (int c = 64 * i; c < 64 * i + 64; c += 4) {
#pragma unroll
                for (int q = 0; q < 2; ++q)
                  mc[q] = fmax3(mc[q], __uint_as_float(sv[c + 2 * q]), __uint_as_float(sv[c + 2 * q + 1]));
              }
              mh[i] = fmaxf(mc[0], mc[1]);
            }
            if constexpr (BIAS)
              raise(fmax3(m_run, fmaf(mh[0], sc, shift[0]), fmaf(mh[1], sc, shift[1])));
            else
              raise(fmaxf(m_run, fmaxf(mh[0], mh[1]) * sc));
            const uint64_t sc2 = f2(sc, sc);
            const uint64_t n0 = f2(shift[0] - m_use, shift[0] - m_use), n1 = f2(shift[1] - m_use, shift[1] - m_use);
            weights([&](int c) {
              const uint64_t s2 = f2(__uint_as_float(sv[2 * c]), __uint_as_float(sv[2 * c + 1]));
              return ffma2(s2, sc2, c < 32 ? n0 : n1);
            });
          }
          if (j > 0) {
            wait(&bar->o_done, (J - 1) & 1);
            tc_fence_after();
            if (__any_sync(0xffffffffu, rescale)) {
              uint32_t ov[32];
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                tmem_ld32(trow + kColO + 32 * i, ov);
                tmem_wait_ld();
#pragma unroll
                for (int c = 0; c < 32; ++c) ov[c] = __float_as_uint(__uint_as_float(ov[c]) * alpha);
                tmem_st32(trow + kColO + 32 * i, ov);
              }
            }
          }
          tmem_st32(trow + kColP + 32, *reinterpret_cast<uint32_t(*)[32]>(&pk[32]));
          tmem_wait_st();
          if (pass == 1 && cls != 0) {
            // which rows of V hold a value that is not finite
            const int sp = J % kVStages;
            unsigned char *vt = smem + kOffV + sp * kTile;
            wait(&bar->v_full[sp], (J / kVStages) & 1);
            for (int r = warp; r < 4; r += vb->active) {
              const uint32_t *vr = reinterpret_cast<const uint32_t *>(vt + (32 * r + lane) * 128);
              bool inf = false;
#pragma unroll 1
              for (int i = 0; i < 32; ++i) {
                const uint32_t y = vr[(i + lane) & 31];
                inf |= (y & 0x7f80u) == 0x7f80u || (y & 0x7f800000u) == 0x7f800000u;
              }
              const uint32_t bits = __ballot_sync(0xffffffffu, inf);
              if (lane == 0) *reinterpret_cast<volatile uint32_t *>(&bar->vflag[r]) = bits;
            }
            meet();
            const volatile uint32_t *vbad = bar->vflag;
            if ((vbad[0] | vbad[1] | vbad[2] | vbad[3]) != 0) {
              // they go to the rows that see them, and out of the tile
              const int t = vb->qi * 128 + tid;
              const bool there = t < p.Nq;
              int row_doc = 0, row_order = 0;
              if (p.q_doc) row_doc = there ? __ldg(p.q_doc + (long long)vb->b * p.Nq + t) : -1;
              if (p.q_order) row_order = there ? __ldg(p.q_order + (long long)vb->b * p.Nq + t) : 0;
              if (row_doc < 0) row_doc = -2;
              uint32_t ov[32];
#pragma unroll 1
              for (int i = 0; i < 2; ++i) {
                if (j > 0) {
                  tmem_ld32(trow + kColO + 32 * i, ov);
                  tmem_wait_ld();
                } else {
#pragma unroll
                  for (int c = 0; c < 32; ++c) ov[c] = 0;
                }
#pragma unroll 1
                for (int u = 0; u < 128; ++u) {
                  if (!(vbad[u >> 5] >> (u & 31) & 1) || code == kNone) continue;
                  if (code == kMixed && (m_doc[u] != row_doc || m_order[u] > row_order)) continue;
#pragma unroll
                  for (int c = 0; c < 32; ++c) {
                    const int d = 32 * i + c;
                    const uint32_t bits = *reinterpret_cast<const uint16_t *>(
                        vt + u * 128 + (((d >> 3) ^ (u & 7)) << 4) + (d & 7) * 2);
                    if ((bits & 0x7f80u) == 0x7f80u)
                      ov[c] = __float_as_uint(__uint_as_float(ov[c]) + __uint_as_float(bits << 16));
                  }
                }
                __syncwarp();
                tmem_st32(trow + kColO + 32 * i, ov);
              }
              tmem_wait_st();
              if (j == 0 && lane == 0) *reinterpret_cast<volatile int *>(&bar->o_init) = 1;
              meet();
              for (int r = warp; r < 4; r += vb->active) {
                uint16_t *vr = reinterpret_cast<uint16_t *>(vt + (32 * r + lane) * 128);
#pragma unroll 1
                for (int c = 0; c < 64; ++c)
                  if ((vr[c] & 0x7f80u) == 0x7f80u) vr[c] = 0;
              }
              fence_async_shared();
            }
            meet();  // the flags have been read
          }
          tc_fence_before();
          __syncwarp();
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          if (lane == 0) mbar_arrive(&bar->p_full);
        }
        const int t = vb->qi * 128 + tid;
        const long long slot = ((long long)vb->bh * p.nq + vb->qi) * p.splits + blockIdx.y;
        if (ok) wait(&bar->o_done, ((pass + 1) * vb->tiles - 1) & 1);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) {
          report_error(p.dev_err, RESS_ERR_DEVICE_TIMEOUT);
          *abort = 1;
          if (p.splits > 1 && t < p.Nq) p.part_ml[slot * 128 + tid] = make_float2(0.f, -1.f);
        } else {
          tc_fence_after();
          uint32_t o[64];
          tmem_ld32(trow + kColO, *reinterpret_cast<uint32_t(*)[32]>(&o[0]));
          tmem_ld32(trow + kColO + 32, *reinterpret_cast<uint32_t(*)[32]>(&o[32]));
          tmem_wait_ld();
          if (masked && pass == 0 && t < p.Nq && l_run != 0.f) {
#pragma unroll
            for (int c = 0; c < 64; ++c) again |= (o[c] & 0x7f800000u) == 0x7f800000u;
          }
          if (t < p.Nq && p.splits > 1) {
            p.part_ml[slot * 128 + tid] = make_float2(m_run, l_run);
            uint4 *dst = reinterpret_cast<uint4 *>(p.part_o + (slot * 128 + tid) * 64);
#pragma unroll
            for (int c = 0; c < 16; ++c) dst[c] = make_uint4(o[4 * c], o[4 * c + 1], o[4 * c + 2], o[4 * c + 3]);
          } else if (t < p.Nq) {
            // a row that saw no key is zero whatever the products hold
            const bool none = l_run == 0.f;
            const float inv = 1.0f / l_run;
            uint32_t w[32];
#pragma unroll
            for (int c = 0; c < 32; ++c)
              w[c] = none ? 0u : pack_bf16x2(__uint_as_float(o[2 * c]) * inv, __uint_as_float(o[2 * c + 1]) * inv);
            uint4 *dst = reinterpret_cast<uint4 *>(p.out + ((size_t)vb->bh * p.Nq + t) * 64);
#pragma unroll
            for (int c = 0; c < 8; ++c) dst[c] = make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
            if (p.lse)
              p.lse[(size_t)vb->bh * p.Nq + t] = none ? -INFINITY : (m_run + __log2f(l_run)) * kLn2;
          }
        }
      }
      if (!masked || pass == 1) break;
      tc_fence_before();
      if (!__syncthreads_or(again)) break;
      tc_fence_after();
    }
  } else if (warp < 4 && t < p.Nq) {
    if (p.splits > 1) {
      p.part_ml[(item * p.splits + blockIdx.y) * 128 + tid] = make_float2(kNoMax, any_bad ? -1.f : 0.f);
    } else if (!any_bad) {
      // nothing to see: zero rows
      uint4 *dst = reinterpret_cast<uint4 *>(p.out + ((size_t)bh * p.Nq + t) * 64);
#pragma unroll
      for (int c = 0; c < 8; ++c) dst[c] = make_uint4(0, 0, 0, 0);
      if (p.lse) p.lse[(size_t)bh * p.Nq + t] = -INFINITY;
    }
  }
  if (tid == kProducerWarp * 32) mbar_wait(&bar->q_full, 0, nullptr);  // whatever became of the row
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(tmem, kTmemCols);
}

// ------------------------------------------------------------------------ join
// One warp per query row: out = sum_s 2^(m_s - m) O_s / sum_s 2^(m_s - m) l_s.  A split with
// l = 0 saw no key (its O is not written); one with l < 0 met an error and leaves the row
// as it was.  A lane weighs a split, so that the O's loads depend on nothing but the weights.
__global__ void __launch_bounds__(256) join_kernel(const float *part_o, const float2 *part_ml, int splits, int nq,
                                                   int Nq, long long rows, __nv_bfloat16 *out, float *lse) {
  wait_prerequisites();
  const long long row = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (row >= rows) return;
  const long long bh = row / Nq;
  const int t = (int)(row - bh * Nq);
  const long long slot0 = (bh * nq + (t >> 7)) * splits;
  const int r = t & 127;
  float m = kNoMax;
  bool bad = false;
  for (int s = lane; s < splits; s += 32) {
    const float2 ml = part_ml[(slot0 + s) * 128 + r];
    m = fmaxf(m, ml.x);
    bad |= ml.y < 0.f;
  }
  if (__any_sync(0xffffffffu, bad)) return;
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  float l = 0.f, o0 = 0.f, o1 = 0.f;
  for (int s0 = 0; s0 < splits; s0 += 32) {
    const int n = min(32, splits - s0);
    float w = 0.f;
    bool some = false;
    if (lane < n) {
      const float2 ml = part_ml[(slot0 + s0 + lane) * 128 + r];
      some = ml.y != 0.f;
      w = some ? ex2_approx(ml.x - m) : 0.f;
      l += w * ml.y;
    }
    const uint32_t mask = __ballot_sync(0xffffffffu, some);
    const float *src = part_o + ((slot0 + s0) * 128 + r) * 64 + 2 * lane;
#pragma unroll 8
    for (int s = 0; s < n; ++s) {
      const float ws = __shfl_sync(0xffffffffu, w, s);
      float2 v = make_float2(0.f, 0.f);
      if (mask >> s & 1) v = *reinterpret_cast<const float2 *>(src + (long long)s * 128 * 64);
      o0 += ws * v.x;
      o1 += ws * v.y;
    }
  }
  for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  const bool none = l == 0.f;
  const float inv = 1.0f / l;
  reinterpret_cast<uint32_t *>(out + row * 64)[lane] = none ? 0u : pack_bf16x2(o0 * inv, o1 * inv);
  if (lse && lane == 0) lse[row] = none ? -INFINITY : (m + __log2f(l)) * kLn2;
}

// ------------------------------------------------------------------- block summaries
// One warp per key block, over its tokens: {min doc, max doc, min order, max order}, and
// {min, max, first position, step} with the step kUneven unless every position is first +
// step * place (a block short of tokens is uneven: it has no last column to measure from).
__global__ void __launch_bounds__(256) summary_kernel(const int32_t *__restrict__ doc,
                                                      const int32_t *__restrict__ order,
                                                      const int32_t *__restrict__ pos, int N, int nk, int kb,
                                                      long long blocks, int4 *__restrict__ out) {
  launch_dependents();
  const long long i = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (i >= blocks) return;
  const long long b = i / nk;
  const int j = (int)(i - b * nk), u0 = j * kb, n = min(N - u0, kb);
  if (doc || order) {
    int4 s = make_int4(INT_MAX, INT_MIN, INT_MAX, INT_MIN);
    for (int u = lane; u < n; u += 32) {
      const int d = doc ? doc[b * N + u0 + u] : 0, o = order ? order[b * N + u0 + u] : 0;
      s.x = min(s.x, d);
      s.y = max(s.y, d);
      s.z = min(s.z, o);
      s.w = max(s.w, o);
    }
    s.x = __reduce_min_sync(0xffffffffu, s.x);
    s.y = __reduce_max_sync(0xffffffffu, s.y);
    s.z = __reduce_min_sync(0xffffffffu, s.z);
    s.w = __reduce_max_sync(0xffffffffu, s.w);
    if (lane == 0) out[i] = s;
  }
  if (pos) {
    pos += b * N + u0;
    int lo = INT_MAX, hi = INT_MIN;
    const long long first = pos[0], step = n > 1 ? pos[1] - first : 0;
    bool even = n == kb && step > -(1 << 20) && step < (1 << 20);
    for (int u = lane; u < n; u += 32) {
      const int x = pos[u];
      lo = min(lo, x);
      hi = max(hi, x);
      even = even && x == first + step * u;
    }
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    even = __all_sync(0xffffffffu, even);
    if (lane == 0) out[blocks + i] = make_int4(lo, hi, (int)first, even ? (int)step : kUneven);
  }
}

// Rows of a masked call, one warp each: how many of the row's kept blocks some query sees, for
// a launch order of the longest rows first.
__global__ void __launch_bounds__(256) plan_kernel(const __grid_constant__ Params p, long long rows,
                                                   int32_t *count) {
  launch_dependents();
  wait_prerequisites();
  const long long item = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (item >= rows) return;
  const long long bh = item / p.nq;
  const int qi = (int)(item - bh * p.nq), b = (int)(bh / p.H);
  int dmin = INT_MAX, dmax = INT_MIN, omax = INT_MIN;
  for (int t = qi * 128 + lane; t < min(p.Nq, qi * 128 + 128); t += 32) {
    const int d = p.q_doc ? p.q_doc[(long long)b * p.Nq + t] : 0;
    if (d < 0) continue;
    dmin = min(dmin, d);
    dmax = max(dmax, d);
    if (p.q_order) omax = max(omax, p.q_order[(long long)b * p.Nq + t]);
  }
  dmin = __reduce_min_sync(0xffffffffu, dmin);
  dmax = __reduce_max_sync(0xffffffffu, dmax);
  omax = __reduce_max_sync(0xffffffffu, omax);
  const int cnt = p.kv_cnt ? min(p.kv_cnt[item], p.nk) : p.nk;
  int n = 0;
  for (int j = lane; j < cnt; j += 32) {
    const int kb = p.kv_idx ? p.kv_idx[item * p.nk + j] : j;
    if (kb < 0 || kb >= p.nk) continue;
    const int4 s = p.blocks[(long long)b * p.nk + kb];
    const bool doc = !p.q_doc || (dmax >= 0 && s.y >= 0 && max(s.x, 0) <= dmax && s.y >= dmin);
    n += doc && (!p.q_order || s.z <= omax);
  }
  n = __reduce_add_sync(0xffffffffu, n);
  if (lane == 0) count[item] = n;
}

// Up to kRankRows rows in descending order of their counts, equal ones by index: every row
// counts those before it, four lanes a row, 64 rows a CTA.  A new view over 32 views (176 rows
// of 687 blocks) takes 183 us with it and 191 with the sort by counters; 1376 rows of 86
// blocks 209 and 203, so it ends at 1024.
constexpr int kRankRows = 1024, kRankRowsOfCta = 64;
__global__ void __launch_bounds__(256) rank_kernel(const int32_t *count, int n, int32_t *order) {
  __shared__ __align__(16) int all[kRankRows + 16];
  launch_dependents();
  wait_prerequisites();
  const int padded = (n + 15) & ~15;
  for (int i = threadIdx.x; i < padded; i += 256) all[i] = i < n ? count[i] : INT_MIN;
  __syncthreads();
  const int i = blockIdx.x * kRankRowsOfCta + (threadIdx.x >> 2), part = threadIdx.x & 3;
  const int own = i < n ? all[i] : 0;
  int rank = 0;
  for (int j = 4 * part; j < padded; j += 16) {
    const int4 c = *reinterpret_cast<const int4 *>(&all[j]);
    rank += (c.x > own || (c.x == own && j < i)) + (c.y > own || (c.y == own && j + 1 < i)) +
            (c.z > own || (c.z == own && j + 2 < i)) + (c.w > own || (c.w == own && j + 3 < i));
  }
  rank += __shfl_xor_sync(0xffffffffu, rank, 1);
  rank += __shfl_xor_sync(0xffffffffu, rank, 2);
  if (i < n && part == 0) order[rank] = i;
}

// Rows of a problem without keys: zero, and lse = -inf.
__global__ void __launch_bounds__(256) no_keys_kernel(long long rows, uint4 *__restrict__ out,
                                                      float *__restrict__ lse) {
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < rows * 8; i += (long long)gridDim.x * 256) {
    out[i] = make_uint4(0, 0, 0, 0);
    if (lse && (i & 7) == 0) lse[i >> 3] = -INFINITY;
  }
}

// CTAs that share a row: as many as keep the whole card (two per SM) busy, each with a few
// tiles of the longest possible row; long rows (16 tiles a part) are split on into up to four
// times as many, since kept lists and masks make them uneven.  A part's sums cost 32 KB each
// way and the join a dependent launch: 4 heads of 1024 tokens, causal with a prefix, 16.6 us
// at 2 tiles a part, 17.8 at 4, 19.0 unsplit; a new view over 32 views 315 us unsplit, 215 at
// four parts (before the order below).
constexpr int kSlots = 2 * 148, kTilesPerSplit = 2, kTilesOfUneven = 16;
int splits_of(const Dims &d, int nq) {
  const long long items = d.BH() * nq;
  const int tiles = (int)((d.N + 127) / 128);
  if (items == 0) return 1;
  long long n = std::max(1ll, std::min(kSlots / items, (long long)(tiles / kTilesPerSplit)));
  while (items * n * 2 <= 4 * kSlots && tiles >= 2 * n * kTilesOfUneven) n *= 2;
  return (int)n;
}

// Rows of masked calls and of kept lists are put in order, longest first, where they come in
// more than one wave and are long enough for the tail to matter (one or two small kernels
// of 3-6 us).
bool plans_order(const Dims &d, int nq) {
  const long long items = d.BH() * nq;
  return items * splits_of(d, nq) > kSlots && items * ((d.N + 127) / 128) >= 64 * kSlots;
}

size_t round256(size_t n) { return (n + 255) & ~(size_t)255; }

// A launch that may overlap the end of the kernel before it (`after`: one of this call's).
template <typename... Sig, typename... Args>
cudaError_t launch_after(void (*kernel)(Sig...), dim3 grid, int threads, size_t smem, cudaStream_t st, bool after,
                         Args... args) {
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = after ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<Sig>(args)...);
}

using KernelFn = void (*)(const CUtensorMap, const CUtensorMap, const CUtensorMap, const Params);
template <int KB>
KernelFn pick(bool cap, bool bias) {
  return cap ? (bias ? masked_attn_kernel<KB, true, true> : masked_attn_kernel<KB, true, false>)
             : (bias ? masked_attn_kernel<KB, false, true> : masked_attn_kernel<KB, false, false>);
}

}  // namespace

size_t masked_attn_workspace_bytes(const Dims &d, int q_len) {
  if (masked_step_fits(d, q_len)) return 0;
  const int nq = (q_len + 127) / 128;
  const int splits = splits_of(d, nq);
  size_t n = plans_order(d, nq) ? 2 * round256(sizeof(int32_t) * (size_t)d.BH() * nq) : 0;
  n += round256(2 * sizeof(int4) * (size_t)d.B * d.nk);
  if (splits > 1)
    n += round256((size_t)d.BH() * nq * splits * 128 * 64 * sizeof(float)) +
         round256((size_t)d.BH() * nq * splits * 128 * sizeof(float2));
  return n;
}

cudaError_t launch_masked_attn(const Dims &d, const MaskedAttnLaunch &a, cudaStream_t st) {
  const ress_attn_mods &m = a.mods;
  const int Nq = m.q_len, nq = (Nq + 127) / 128;
  const long long rows = d.BH() * Nq;
  if (d.N == 0) {
    const long long ctas = std::min((rows * 8 + 255) / 256, 4096ll);
    no_keys_kernel<<<(unsigned)ctas, 256, 0, st>>>(rows, static_cast<uint4 *>(a.out), a.lse);
    return cudaGetLastError();
  }
  if (masked_step_fits(d, Nq)) return launch_masked_step(d, a, st);
  CUtensorMap mq, mk, mv;
  if (!make_map(&mq, a.q, Nq, d.BH(), 128) || !make_map(&mk, a.k, d.N, d.BH(), d.kb) ||
      !make_map(&mv, a.v, d.N, d.BH(), d.kb))
    return cudaErrorNotSupported;
  Params p = {};
  p.kv_idx = a.kv_idx;
  p.kv_cnt = a.kv_cnt;
  if (m.slopes) {
    p.slopes = m.slopes;
    p.q_pos = m.q_pos;
    p.k_pos = m.k_pos;
  }
  p.q_doc = m.q_doc;
  p.k_doc = m.k_doc;
  p.q_order = m.q_order;
  p.k_order = m.k_order;
  p.out = static_cast<__nv_bfloat16 *>(a.out);
  p.lse = a.lse;
  p.dev_err = a.dev_err;
  p.B = d.B;
  p.H = d.H;
  p.N = d.N;
  p.Nq = Nq;
  p.nq = nq;
  p.nk = d.nk;
  p.splits = splits_of(d, nq);
  // rows in parts are few, or put in order below; a caller's order that left one out would
  // leave its parts unwritten for the join
  p.order = p.splits == 1 ? a.order : nullptr;
  p.scale_log2 = a.scale * kLog2e;
  p.cap_log2 = m.softcap * kLog2e;
  p.cap_in = m.softcap > 0.f ? a.scale / m.softcap : 0.f;
  p.cap_half = 0.5f / p.cap_in;
  // The fused cap: its coefficients, scale (scale / c)^2i times the fit's, must be normal fp32
  // numbers, and the bound that it takes for the row's maximum may lie 2 |z| above it, which
  // costs the exponents that range: 64 at most.
  p.cap_a = -1.f;
  if (p.cap_in > 1e-5f && p.cap_in < 1e5f) {
    bool normal = true;
    double k = (double)p.cap_log2 * p.cap_in;
    for (int i = 0; i < 4; ++i, k *= (double)p.cap_in * p.cap_in) {
      const double x = std::abs(kTanhFit3[i] * k);
      normal = normal && x >= FLT_MIN && x <= FLT_MAX;
      p.cap_k[i] = normal ? (float)(kTanhFit3[i] * k) : 0.f;
    }
    if (normal) p.cap_a = std::min(0.375f / p.cap_in, 32.f / p.scale_log2);
  }
  unsigned char *ws = static_cast<unsigned char *>(a.workspace);
  int4 *blocks = reinterpret_cast<int4 *>(ws);
  p.blocks = blocks;
  const long long items = d.BH() * nq;
  ws += round256(2 * sizeof(int4) * (size_t)d.B * d.nk);
  int32_t *count = nullptr, *sorted = nullptr;
  if (plans_order(d, nq)) {
    count = reinterpret_cast<int32_t *>(ws);
    sorted = reinterpret_cast<int32_t *>(ws + round256(sizeof(int32_t) * (size_t)items));
    ws += 2 * round256(sizeof(int32_t) * (size_t)items);
  }
  if (p.splits > 1) {
    p.part_o = reinterpret_cast<float *>(ws);
    ws += round256((size_t)items * p.splits * 128 * 64 * sizeof(float));
    p.part_ml = reinterpret_cast<float2 *>(ws);
  }
  if (m.q_doc || m.q_order || m.slopes) {
    const long long n = 1ll * d.B * d.nk;
    summary_kernel<<<(unsigned)((n + 7) / 8), 256, 0, st>>>(m.k_doc, m.k_order, p.k_pos, d.N, d.nk, d.kb, n,
                                                            blocks);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  const bool masked = m.q_doc || m.q_order;
  if (sorted && !p.order && (masked || p.kv_cnt)) {
    if (masked) {
      cudaError_t e = launch_after(plan_kernel, dim3((unsigned)((items + 7) / 8)), 256, 0, st, true, p, items, count);
      if (e != cudaSuccess) return e;
    }
    const int32_t *by = masked ? count : p.kv_cnt;
    cudaError_t e;
    if (items <= kRankRows) {
      const unsigned ctas = (unsigned)((items + kRankRowsOfCta - 1) / kRankRowsOfCta);
      e = launch_after(rank_kernel, dim3(ctas), 256, 0, st, masked || m.slopes, by, (int)items, sorted);
    } else {
      Dims rows = d;
      rows.nb = rows.nq = nq;
      e = launch_schedule(rows, by, sorted, st);
    }
    if (e != cudaSuccess) return e;
    p.order = sorted;
  }
  KernelFn kern = d.kb == 64 ? pick<64>(m.softcap > 0.f, m.slopes != nullptr)
                             : pick<128>(m.softcap > 0.f, m.slopes != nullptr);
  cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void *>(kern),
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  if (e != cudaSuccess) return e;
  e = launch_after(kern, dim3((unsigned)items, (unsigned)p.splits), kThreads, kSmemBytes, st,
                   masked || m.slopes || (sorted && p.order == sorted), mq, mk, mv, p);
  if (e != cudaSuccess || p.splits == 1) return e;
  return launch_after(join_kernel, dim3((unsigned)((rows + 7) / 8)), 256, 0, st, true, (const float *)p.part_o,
                      (const float2 *)p.part_ml, p.splits, nq, Nq, rows, p.out, p.lse);
}

}  // namespace ress
