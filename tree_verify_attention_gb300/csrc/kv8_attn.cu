// Attention of the draft-tree nodes (one node: plain decode) over the 8-bit
// cache, in two launches: the attention over slices of the keys, and the
// merge of the slices.
//
//   out[i][h] = sum_j softmax_j(scale q . k_j) v_j   over the keys visible to
//   node i: complete blocks (8-bit codes), the open block's bf16 rows, and
//   the tree rows of the node and its ancestors.
//
// Keys are the M dimension of both products, so that few query rows cost
// little and no code is dequantised twice:
//
//   S^T [128 keys x R rows]  = K^ [128 x D] Q^T      A = K^ in TMEM
//   O^T [D x R rows]        += V^T [D x 128] P^T     A = V^T in TMEM
//
// A warp turns its 32 keys' (K) or 32 dims' (V) codes into binary16 integers
// (exact) in registers and stores them straight into TMEM: the cache's layout
// puts them there as consecutive 16-byte pieces, and the operands never touch
// shared memory. Q^T and P^T are the small B operands in shared memory.
//
// Scales never multiply a code. Lane = key, so a key's K scale is one factor
// of its thread, a_j = k_scale * softmax scale * log2 e; its V scale goes into
// the exponent,
//
//   P'_jc = 2^(S_jc a_j + log2 v_scale_j - m_c),   O += P' code,
//   l_c  += P'_jc / v_scale_j                      (f32, per thread)
//
// with m_c a reference of the column, not its exact maximum: a chunk only has
// to show that no P' passes 2^15 (what binary16 holds), which one vote decides;
// columns' maxima are reduced across lanes only when one does. A new reference
// puts the largest P' so far at 2^8, not at 1: binary16 then keeps its full
// 2^-11 for contributions down to 2^-22 of it (a key that takes nearly all of
// the weight and adds nothing leaves the output to such ones), and smaller
// ones are within 2^-33 of it.
// The tail and tree rows (bf16) are one last chunk of at most 63 + 65 = 128
// keys, scaled by a power of two per key to binary16 range, so that it runs
// through the same products with its own a_j and v_scale_j. Q is scaled by one
// power of two per tile while the tile's rows lie within 2^10 of each other;
// else each row has its own and the difference becomes a factor of the column
// ("wide" units, which a row of garbage beside ordinary ones leads to). Every
// operand is then exact in binary16 but P', whose rounding (2^-11 of each
// weight, the normaliser has none) is below that of the bf16 output; a float32
// output is as exact as its weights. (Elements below 2^-21 of their row's
// largest are not exact either: they are within 2^-29 of that one.)
//
// Roles of a CTA (one per SM): 8 or 16 softmax warps (lane quadrant w % 4,
// column group w / 4), four warps that put K codes into TMEM, four for V, one
// that issues MMAs, two that copy K and V. A unit is (KV head, tile of at most
// 80 query rows, or 96 below D = 256, slice of the chunks). Bound by HBM while
// a tile has few rows, by the softmax and the conversion for many: 24 heads of
// 256 over 131072 positions take 48.9 us for one node (5.5 TB/s) and 99 us for
// 23 (750 TFLOP/s; 71 % of the issue slots busy).

#include <atomic>
#include <math.h>
#include <type_traits>

#include "kv8.cuh"
#include "tc.cuh"
#include "tmem_io.cuh"

namespace dfv {

constexpr int kAtKeys = 128;         // keys of a chunk
constexpr int kTreeCost = 6;         // chunks that the bf16 chunk counts as
constexpr float kTop = 8.0f;         // exponent of the largest P' under a new reference
constexpr float kRaise = 15.0f;      // a larger exponent moves the reference
constexpr float kNoRef = 3e38f;      // -reference of a column that has seen no key
constexpr float kFar = 262144.0f;    // a larger reference is kept in two parts
// V scale that a key without any value counts with: it adds nothing to the
// output, so its weight must not make the others' small (its sum of up to 2^17
// keys of 2^15 / kNoValue stays in float32).
constexpr float kNoValue = 8.0779357e-28f;   // 2^-90
constexpr int kSpread = 10;          // log2 of the ratio of rows that share a scale
constexpr uint32_t kNotFinite = 0x10000u;   // in a row's magnitude: it holds inf or NaN
constexpr float kLog2eF = 1.4426950408889634f;
constexpr float kLn2F = 0.6931471805599453f;

template <int D, int R>
struct AttnShape {
  // Softmax warps: four lane quadrants times the column groups. The softmax
  // of many columns is a long chain per warp; twice the warps, with half the
  // columns each, shorten it and leave 72 registers a thread (23 nodes, ctx
  // 131072: 127 -> 120 us; 12 warps of 24 columns were no better than 16).
  static constexpr int kSoft = R >= 64 ? 16 : 8;
  static constexpr int kGroups = kSoft / 4;
  static constexpr int kCols = R / kGroups;             // columns of a softmax thread
  static constexpr int kThreads = (kSoft + 11) * 32;
  static constexpr int kHalves = D == 256 ? 2 : 1;      // 128-lane parts of V^T
  // K^ and V^ are handed to the products in parts of kPart columns (two per
  // operand at D = 256 and 128): the next chunk's part can be written while
  // the products read the other
  static constexpr int kPart = D == 256 ? 64 : 32;
  static constexpr int kKSub = D / 2 / kPart, kVSub = 64 * kHalves / kPart;
  static constexpr int kRaw = kAtKeys * D;              // bytes of a chunk's K (V) codes
  static constexpr int kRowB = D * 2 + 16;              // a staged bf16 row (padded: banks)
  static constexpr int kPBlk = (R + 63) / 64;
  static constexpr int kPBytes = kPBlk * kAtKeys * 128;
  static constexpr int kPBufs = R <= 64 || D < 256 ? 2 : 1;
  static constexpr int kStages = D == 256 ? 2 : 4;
  static constexpr int kQBytes = R * D * 2;
  static constexpr int kRing = kStages * 2 * kRaw;
  static constexpr int kRows = 2 * kAtKeys * kRowB;
  static constexpr int kOffQ = ((kRing > kRows ? kRing : kRows) + 1023) / 1024 * 1024;
  static constexpr int kOffP = (kOffQ + kQBytes + 1023) / 1024 * 1024;
  static constexpr int kBytes = kOffP + kPBufs * kPBytes + 1024;
  // TMEM columns
  static constexpr uint32_t kTK = 0;
  static constexpr uint32_t kTV = kTK + D / 2;
  static constexpr uint32_t kTS = kTV + 64 * kHalves;
  static constexpr uint32_t kTO = kTS + R;
  static_assert(kTO + R * kHalves <= 512, "TMEM columns");
  static_assert(kBytes <= 219 * 1024, "shared memory");
};

struct AttnParams {
  dfv_kv8_cache c;
  int nblk;
  int n_nodes, max_depth, hq, group, window;
  uint32_t group_m;                 // ceil(2^32 / group): r / group = umulhi(r, group_m)
  int rows_tile, rows;              // query rows of a tile, of a KV head
  const __nv_bfloat16* q;
  const __nv_bfloat16* tree_k;
  const __nv_bfloat16* tree_v;
  const int32_t* parent;
  float scale;
  float* part_o;     // [head][tile][split][R][D], normalised
  float* part_lse;   // [head][tile][split][R], base 2
  uint32_t* status;
};

// 16 codes as 8 words of binary16 pairs: 0x6400 | u is 1024 + u, and u = code + 128.
__device__ __forceinline__ void codes_to_half(const uint4& v, uint32_t* w) {
  const uint32_t in[4] = {v.x, v.y, v.z, v.w};
  const __half2 bias = __float2half2_rn(1152.0f);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t u = in[k] ^ 0x80808080u;
    const uint32_t lo = __byte_perm(u, 0x64646464u, 0x4140);
    const uint32_t hi = __byte_perm(u, 0x64646464u, 0x4342);
    const __half2 a = __hsub2(*reinterpret_cast<const __half2*>(&lo), bias);
    const __half2 b = __hsub2(*reinterpret_cast<const __half2*>(&hi), bias);
    w[2 * k] = *reinterpret_cast<const uint32_t*>(&a);
    w[2 * k + 1] = *reinterpret_cast<const uint32_t*>(&b);
  }
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float lg2_fast(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A packed pair of bf16 values times f, as a pair of binary16 values.
__device__ __forceinline__ uint32_t scaled_half2(uint32_t bf, float f) {
  return pack_half2(__uint_as_float(bf << 16) * f, __uint_as_float(bf & 0xFFFF0000u) * f);
}

// Largest magnitude (bf16 bits) of a staged row of D values.
template <int D>
__device__ __forceinline__ uint32_t row_max(const uint8_t* row) {
  uint32_t m = 0;
#pragma unroll 8
  for (int j = 0; j < D / 8; ++j) {
    const uint4 v = *reinterpret_cast<const uint4*>(row + j * 16);
    m = __vmaxu2(m, __vmaxu2(__vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu),
                             __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu)));
  }
  return max(m & 0xFFFFu, m >> 16);
}

template <int D, int R>
__global__ void __launch_bounds__(AttnShape<D, R>::kThreads, 1)
    kv8_attn_kernel(const __grid_constant__ AttnParams p) {
  using A = AttnShape<D, R>;
  constexpr int HC = A::kCols, SW = A::kSoft, NG = A::kGroups;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* sQ = smem + A::kOffQ;
  uint8_t* sP = smem + A::kOffP;
  // raw codes landed / read (per stage); operand part written / read by the
  // products (K's last part read: the scores are there); scores read; P
  // written and O there (two each, used in turn: a phase's parity tells it
  // from its neighbours only, and the softmax may lag P V by two chunks);
  // bf16 rows landed, and their scales written (once: the operands' own
  // phases may be one behind or ahead of the softmax here)
  __shared__ uint64_t b_kraw[4], b_kdone[4], b_vraw[4], b_vdone[4];
  __shared__ uint64_t b_khat[4], b_kfree[4], b_vhat[4], b_vfree[4];
  __shared__ uint64_t b_sfree, b_q, b_end, b_krow, b_vrow, b_rowsc, b_sc, b_p[2],
      b_pv[2];
  __shared__ uint32_t s_tmem;
  __shared__ volatile int s_dead;
  __shared__ int s_parent[kMaxNodes], s_maxdepth;
  // columns (of each group) that see a tree node; columns by depth, and up to a depth
  __shared__ uint32_t s_see[kMaxNodes][NG], s_dep[kMaxNodes][NG], s_upto[kMaxNodes][NG];
  // -(reference), and in a wide unit its second part and the column's factor
  __shared__ __align__(16) float s_neg[R], s_f[R], s_lo[R], s_cf[R];
  __shared__ float s_red[4][R];
  // (K scale, log2 and inverse of the V scale) of the blocks of two times 16 chunks
  __shared__ __align__(16) float4 s_sc[64];
  __shared__ float s_ksc[kAtKeys];
  __shared__ __align__(8) float s_vfac[kAtKeys];
  __shared__ int s_vexp[kAtKeys];
  __shared__ uint8_t s_bad[2][kAtKeys];
  __shared__ uint32_t s_qmax, s_qmin;   // largest and smallest of the rows' magnitudes

  const int tid = threadIdx.x, lane = tid & 31;
  // both the same in every lane, which the compiler knows of a reduction's
  // result: what follows from them then lives in uniform registers
  const int warp =
      static_cast<int>(__reduce_max_sync(0xFFFFFFFFu, static_cast<unsigned>(tid >> 5)));
  // what touches no global memory may run under the kernel before
  if (warp == SW + 9 && lane == 0) {
    for (int s = 0; s < 4; ++s) {
      mbar_init(&b_kraw[s], 1);
      mbar_init(&b_vraw[s], 1);
      mbar_init(&b_kdone[s], 4);
      mbar_init(&b_vdone[s], 4);
      mbar_init(&b_khat[s], 4);
      mbar_init(&b_vhat[s], 4);
      mbar_init(&b_kfree[s], s == A::kKSub - 1 ? 2 : 1);
      mbar_init(&b_vfree[s], 1);
    }
    mbar_init(&b_sfree, SW);
    mbar_init(&b_q, SW);
    mbar_init(&b_end, 1);
    mbar_init(&b_krow, 1);
    mbar_init(&b_vrow, 1);
    mbar_init(&b_rowsc, 8);
    mbar_init(&b_sc, 1);
    for (int k = 0; k < 2; ++k) {
      mbar_init(&b_p[k], SW);
      mbar_init(&b_pv[k], 1);
    }
    fence_mbar_init();
  }
  if (tid == 0) {
    s_dead = 0;
    s_qmax = 0;
    s_qmin = kNotFinite;
    s_maxdepth = 0;
  }
  const int split = blockIdx.x, splits = gridDim.x, tile = blockIdx.y, h = blockIdx.z;
  const int row0 = tile * p.rows_tile, n_rows = min(p.rows_tile, p.rows - row0);
  grid_dep_wait();
  grid_dep_launch_dependents();   // the merge may be set up (after the wait: see common.cuh)
  // Not before the wait: a kernel that has let this one start may allocate its
  // own columns only after that, and would wait for these for ever.
  if (warp == SW + 8) tc::tmem_alloc(&s_tmem, 512);
  int C = __reduce_max_sync(0xFFFFFFFFu, p.c.state[0]);
  const int held = p.c.state[2];
  for (int i = tid; i < p.n_nodes; i += A::kThreads) {
    int pa = i == 0 ? -1 : p.parent[i];
    if (i > 0 && (pa < 0 || pa >= i)) {
      report(p.status, DFV_DEV_BAD_TREE);
      pa = 0;
    }
    s_parent[i] = pa;
#pragma unroll
    for (int g = 0; g < NG; ++g) s_see[i][g] = s_dep[i][g] = 0;
  }
  if (C < 0 || C > p.c.capacity || (C % kBlk != 0 && C / kBlk < held)) {
    if (tid == 0) report(p.status, DFV_DEV_CTX);
    C = max(0, min(C, p.c.capacity));
    if (C / kBlk < held) C = C / kBlk * kBlk;   // the tail has other rows there
  }
  // Chunks: complete blocks [fb, open) two at a time, then the bf16 chunk,
  // which belongs to the last slice and counts as several: it waits for its
  // rows when the others already land.
  const int open = C / kBlk, T = C % kBlk;
  const int lo_min = p.window > 0 ? max(0, C - p.window + 1) : 0;
  const int fb = min(lo_min / kBlk, open);
  const int nq = (open - fb + 1) / 2;
  const int per = (nq + kTreeCost) / splits, rem = nq + kTreeCost - per * splits;
  const bool has_tree = split == splits - 1;    // its last chunk is the bf16 one
  const int c0 = min(nq, split * per + split * rem / splits);
  const int n8 = (has_tree ? nq : min(nq, (split + 1) * per + (split + 1) * rem / splits)) - c0;
  const int n = n8 + (has_tree ? 1 : 0);
  const int live_rows = T + p.n_nodes;          // keys of the bf16 chunk

  // raw K (V) codes of chunk i into its stage (one thread)
  auto copy_codes = [&](int i, bool v) {
    const int s = i % A::kStages, b = fb + 2 * (c0 + i);
    const uint32_t bytes = static_cast<uint32_t>(min(2, open - b) * kBlk * D);
    const int64_t off = (static_cast<int64_t>(h) * p.nblk + b) * kBlk * D;
    uint64_t* bar = v ? &b_vraw[s] : &b_kraw[s];
    mbar_arrive_expect_tx(bar, bytes);
    bulk_g2s(smem + (s * 2 + v) * A::kRaw, (v ? p.c.v_codes : p.c.k_codes) + off, bytes, bar);
  };
  // K (V) rows of the bf16 chunk over the ring (one warp)
  auto copy_rows = [&](bool v) {
    uint64_t* bar = v ? &b_vrow : &b_krow;
    if (lane == 0) mbar_arrive_expect_tx(bar, static_cast<uint32_t>(live_rows * D * 2));
    __syncwarp();
    const __nv_bfloat16* tail = static_cast<const __nv_bfloat16*>(v ? p.c.v_tail : p.c.k_tail) +
                                (static_cast<int64_t>(h) * 2 + (open & 1)) * kBlk * D;
    const __nv_bfloat16* tree = (v ? p.tree_v : p.tree_k) + static_cast<int64_t>(h) * D;
    for (int k = lane; k < live_rows; k += 32)
      bulk_g2s(smem + ((v ? kAtKeys : 0) + k) * A::kRowB,
               k < T ? tail + k * D
                     : tree + static_cast<int64_t>(k - T) * p.c.n_kv_heads * D,
               D * 2, bar);
  };

  const int first_copies = min(n8, A::kStages);
  // the copying warps, one for K and one for V: the first copies wait for nothing
  if (warp >= SW + 9) {
    named_sync(1, 64);   // the barriers are there
    fence_proxy_async_global();   // what earlier kernels wrote, to the copy engine
    if (lane == 0)
      for (int i = 0; i < first_copies; ++i) copy_codes(i, warp == SW + 10);
    if (has_tree && n8 == 0) copy_rows(warp == SW + 10);
  }
  // Q rows of the tile, into registers meanwhile (softmax warps)
  constexpr int kQSteps = (R * D / 8 + SW * 32 - 1) / (SW * 32);
  uint4 qv[kQSteps];
  if (warp < SW) {
#pragma unroll
    for (int k = 0; k < kQSteps; ++k) {
      const int it = tid + k * (SW * 32), r = it / (D / 8), j = it % (D / 8);
      qv[k] = make_uint4(0, 0, 0, 0);
      if (r < n_rows) {
        const int node = static_cast<int>(p.group == 1 ? row0 + r : __umulhi(row0 + r, p.group_m));
        const int row = node * p.hq + h * p.group + (row0 + r - node * p.group);
        qv[k] = *reinterpret_cast<const uint4*>(p.q + static_cast<int64_t>(row) * D + j * 8);
      }
    }
  }
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = s_tmem;
  const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;   // quadrant's first lane << 16

  if (warp >= SW + 9) {
    // ------------------------------------------------------ bulk copies
    const bool v = warp == SW + 10;
    uint64_t* raw_full = v ? b_vraw : b_kraw;
    bool ok = true;
    int issued = first_copies;
    // The K warp also prepares the blocks' scales, 32 blocks (16 chunks) at a
    // time, loaded a batch ahead (plain loads, not the read-only path: this
    // kernel may start before the one that wrote them ends) and written before
    // the first copy of their chunks: the softmax reads them after copy,
    // conversion and product S of the chunk, each of which waits for the one
    // before. Only the first batch, written after its copies, has a barrier of
    // its own. The copies are kStages + 3 chunks ahead of the softmax at most,
    // so a batch written in the place of the one before the last finds it read.
    // Against each softmax lane loading its block's scales: 23 nodes at ctx
    // 131072 100.4 for 103.5 us, 65 at ctx 32791 71.3 for 70.6.
    const int64_t sc0 = static_cast<int64_t>(h) * p.nblk + fb + 2 * c0;
    float ks = 0.0f, vs = 0.0f;
    auto load_scales = [&](int batch) {
      const int b = batch * 32 + lane;
      if (fb + 2 * c0 + b < open && b < 2 * n8) {
        ks = p.c.k_scale[sc0 + b];
        vs = p.c.v_scale[sc0 + b];
      }
    };
    auto put_scales = [&](int batch) {
      const float sv = fmaxf(vs, kNoValue);         // (others are 2^-47 at least)
      const float lv = lg2_fast(sv);                // within 2^-20, in both
      s_sc[(batch & 1) * 32 + lane] = make_float4(ks, lv, tc::ex2(-lv), 0.0f);
      __syncwarp();
    };
    if (!v) {
      load_scales(0);
      put_scales(0);
      if (lane == 0) mbar_arrive(&b_sc);
      load_scales(1);
    }
    for (int i = first_copies; ok && i < n8; ++i) {
      ok = role_wait(v ? &b_vdone[i % A::kStages] : &b_kdone[i % A::kStages],
                     (i / A::kStages - 1) & 1, &s_dead);
      ok = __all_sync(0xFFFFFFFFu, ok);
      if (!ok) break;
      if (!v && i % 16 == 0) {
        put_scales(i / 16);
        load_scales(i / 16 + 1);
      }
      if (lane == 0) copy_codes(i, v);
      issued = i + 1;
    }
    if (has_tree && n8 > 0) {
      for (int i = max(0, n8 - A::kStages); ok && i < n8; ++i)
        ok = role_wait(v ? &b_vdone[i % A::kStages] : &b_kdone[i % A::kStages],
                       (i / A::kStages) & 1, &s_dead);
      ok = named_sync_and(1, 64, ok);   // both rings have been read
      if (ok) copy_rows(v);
    }
    // copies that nobody waits for any more must still land
    if (s_dead) {
      for (int i = max(0, issued - A::kStages); i < issued; ++i)
        mbar_wait_bounded(&raw_full[i % A::kStages], (i / A::kStages) & 1);
      if (has_tree && ok) mbar_wait_bounded(v ? &b_vrow : &b_krow, 0);
    }
  } else if (warp == SW + 8) {
    // ------------------------------------------------------ MMA issue
    // The whole warp walks the loop and one elected lane issues: the compiler
    // then keeps descriptors in uniform registers. One lane in a divergent
    // branch took 45 to 56 cycles per MMA whatever its size; elected, an MMA
    // takes its R / 2 cycles (11 at R = 16, 40 at R = 80).
    if (n > 0) {
      constexpr uint32_t id_s = tc::idesc_f16(128, R);
      constexpr uint32_t id_o = tc::idesc_f16(128, R, true);
      const uint64_t qd = tc::smem_desc_sw128(smem_u32(sQ), 1024);
      auto all_wait = [&](uint64_t* bar, uint32_t parity) {
        const bool got = __all_sync(0xFFFFFFFFu, role_wait(bar, parity, &s_dead));
        tc::fence_after_sync();
        return got;
      };
      // S^T of chunk i, part by part as K^ arrives. A commit costs about as
      // much as eight MMAs of 16 columns, so there is one for each part: the
      // last one also tells that S is there and that all products before,
      // P V of chunk i - 2 among them, have ended.
      auto issue_s = [&](int i) {
        if (i > 0 && !all_wait(&b_sfree, (i - 1) & 1)) return false;
#pragma unroll
        for (int c = 0; c < A::kKSub; ++c) {
          if (!all_wait(&b_khat[c], i & 1)) return false;
          if (tc::elect_one()) {
#pragma unroll
            for (int kk = c * A::kPart / 8; kk < (c + 1) * A::kPart / 8; ++kk)
              tc::mma_f16_ts(tmem + A::kTS, tmem + A::kTK + kk * 8,
                             qd + static_cast<uint64_t>(((kk >> 2) * R * 128 + (kk & 3) * 32) >> 4),
                             id_s, kk > 0 ? 1u : 0u);
            tc::commit(&b_kfree[c]);
            // (an arrival of its own: a commit orders the products, not the scales)
            if (c == A::kKSub - 1) mbar_arrive(&b_kfree[c]);
          }
          __syncwarp();
        }
        return true;
      };
      bool ok = all_wait(&b_q, 0) && issue_s(0);
      for (int i = 0; ok && i < n; ++i) {
        if (i + 1 < n) ok = issue_s(i + 1);
        const int pb = i & 1;
        ok = ok && all_wait(&b_p[pb], (i >> 1) & 1);
        const uint64_t pd = tc::smem_desc_sw128_mn(
            smem_u32(sP + (A::kPBufs == 2 ? pb : 0) * A::kPBytes), kAtKeys * 128, 1024);
        // O^T, eight steps of 16 keys for each half of the dims
#pragma unroll
        for (int c = 0; c < A::kVSub; ++c) {
          ok = ok && all_wait(&b_vhat[c], i & 1);
          if (!ok) break;
          if (tc::elect_one()) {
#pragma unroll
            for (int kk = c * A::kPart / 8; kk < (c + 1) * A::kPart / 8; ++kk)
              tc::mma_f16_ts(tmem + A::kTO + (kk >> 3) * R, tmem + A::kTV + kk * 8,
                             pd + static_cast<uint64_t>(((kk & 7) * 16 * 128) >> 4),
                             id_o, i > 0 || (kk & 7) > 0 ? 1u : 0u);
            tc::commit(c == A::kVSub - 1 ? &b_pv[pb] : &b_vfree[c]);
          }
          __syncwarp();
        }
      }
      if (!ok) {
        s_dead = 1;
        // MMAs in flight must end before TMEM is freed
        if (tc::elect_one()) tc::commit(&b_end);
        __syncwarp();
        mbar_wait_bounded(&b_end, 0);
      }
    }
  } else if (warp >= SW) {
    // ------------------------------------------------------ operands to TMEM
    // One body for both operands: the loops of all roles together have to
    // stay in the instruction cache (a body per operand: 110 instead of 107 us
    // for 23 nodes at ctx 131072).
    const bool is_v = warp >= SW + 4;
    const int slot = (warp & 3) * 32 + lane;   // key (K) or dim of a half (V)
    uint64_t* raw_full = is_v ? b_vraw : b_kraw;
    uint64_t* raw_done = is_v ? b_vdone : b_kdone;
    uint64_t* hat = is_v ? b_vhat : b_khat;
    const uint32_t t_op = tmem + lanes + (is_v ? A::kTV : A::kTK);
    constexpr int kPer = A::kPart / 32, kPieces = A::kVSub * kPer;   // pieces of 32 columns
    static_assert(A::kKSub == A::kVSub || (D == 64 && A::kKSub == 1), "parts");
    const int pieces = D == 64 && !is_v ? 1 : kPieces;
    const bool works = !is_v || D >= 128 || slot < D;   // D = 64: V^T has 64 lanes
    // the bytes of a piece, for this thread: K 64 dims of its key (16-byte
    // pieces 64 * 16 apart), V 64 keys of its dim (D * 16 apart); pieces of V
    // run over the chunk's blocks, then the halves of the dims
    const int base0 = is_v ? A::kRaw + slot * 16 : (slot >> 6) * kBlk * D + (slot & 63) * 16;
    const int step = is_v ? D * 16 : kBlk * 16;
    const int step1 = is_v ? kBlk * D : 4 * kBlk * 16, step2 = is_v ? 128 * 16 : 8 * kBlk * 16;
    bool ok = true;
    // A part's columns are free once the products have read the last chunk's.
    auto take = [&](int i, int part) {
      if (i > 0)
        ok = is_v && part == A::kVSub - 1
                 ? role_wait(&b_pv[(i - 1) & 1], ((i - 1) >> 1) & 1, &s_dead)
                 : role_wait(is_v ? &b_vfree[part] : &b_kfree[part], (i - 1) & 1, &s_dead);
      ok = __all_sync(0xFFFFFFFFu, ok);   // the TMEM stores are warp-wide
      tc::fence_after_sync();
    };
    auto give = [&](int part) {
      tc::store_wait();
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&hat[part]);
    };
    for (int i = 0; ok && i < n8; ++i) {
      const int s = i % A::kStages;
      ok = role_wait(&raw_full[s], (i / A::kStages) & 1, &s_dead);
      ok = __all_sync(0xFFFFFFFFu, ok);
      if (!ok) break;
      const uint8_t* raw = smem + s * 2 * A::kRaw + base0;
      uint4 q[4];
      auto fetch = [&](int c) {
        const uint8_t* mine = raw + (c >> 1) * step2 + (c & 1) * step1;
#pragma unroll
        for (int j = 0; j < 4; ++j) q[j] = *reinterpret_cast<const uint4*>(mine + j * step);
      };
      if (works) fetch(0);
#pragma unroll
      for (int c = 0; c < kPieces; ++c) {
        if (c >= pieces) break;
        uint32_t w[32];
        if (works) {
#pragma unroll
          for (int j = 0; j < 4; ++j) codes_to_half(q[j], w + 8 * j);
          if (c + 1 < pieces) fetch(c + 1);   // lands while this piece is handed over
        }
        if (c + 1 == pieces) {   // every code is in registers
          __syncwarp();
          if (lane == 0) mbar_arrive(&raw_done[s]);
        }
        if (c % kPer == 0) {
          // a store takes its time: waited for after the next conversion
          if (c > 0) give(c / kPer - 1);
          take(i, c / kPer);
          if (!ok) break;
        }
        if (works) tc::TmemIo<32>::store(t_op + c * 32, w);
      }
      if (!ok) break;
      give((pieces - 1) / kPer);
    }
    if (has_tree) {
      // The bf16 chunk: key slots [0, T) are the open block's rows, then the
      // tree nodes. Each key is scaled to binary16 by a power of two (largest
      // magnitude in [64, 128)).
      ok = ok && role_wait(is_v ? &b_vrow : &b_krow, 0, &s_dead);
      ok = named_sync_and(is_v ? 3 : 2, 128, ok);
    }
    if (has_tree && ok) {
      uint8_t* rows = smem + (is_v ? kAtKeys * A::kRowB : 0);
      uint8_t* row = rows + slot * A::kRowB;
      const bool live = slot < live_rows;
      const uint32_t m = live ? row_max<D>(row) : 0u;
      const bool bad = m >= kBigBits;   // infinite, NaN or out of range
      const int e = max(static_cast<int>(m >> 7), 86);
      const float f = bad || !live ? 0.0f : pow2i(133 - e);
      s_bad[is_v][slot] = bad;
      if (bad) report(p.status, DFV_DEV_NONFINITE);
      if (!is_v) {
        s_ksc[slot] = bad ? 0.0f : pow2i(e - 133);
      } else {
        s_vexp[slot] = bad ? 0 : m == 0 ? -90 : e - 133;
        s_vfac[slot] = f;
      }
      if (bad || !live) {   // no 0 * inf below
#pragma unroll 1
        for (int j = 0; j < D / 8; ++j)
          *reinterpret_cast<uint4*>(row + j * 16) = make_uint4(0, 0, 0, 0);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&b_rowsc);
      if (is_v) named_sync(3, 128);   // V reads across rows
#pragma unroll 1
      for (int c = 0; c < pieces; ++c) {
        uint32_t w[32];
        if (!is_v) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const uint4 x = *reinterpret_cast<const uint4*>(row + (c * 8 + j) * 16);
            w[4 * j] = scaled_half2(x.x, f);
            w[4 * j + 1] = scaled_half2(x.y, f);
            w[4 * j + 2] = scaled_half2(x.z, f);
            w[4 * j + 3] = scaled_half2(x.w, f);
          }
        } else if (works) {
          const int d = (c >> 1) * 128 + slot, kb = (c & 1) * 64;
          const uint8_t* col = rows + kb * A::kRowB + d * 2;
          const float2* fac = reinterpret_cast<const float2*>(s_vfac + kb);
#pragma unroll
          for (int q = 0; q < 32; ++q) {
            const uint32_t a = *reinterpret_cast<const uint16_t*>(col + 2 * q * A::kRowB);
            const uint32_t b = *reinterpret_cast<const uint16_t*>(col + (2 * q + 1) * A::kRowB);
            const float2 g = fac[q];
            w[q] = pack_half2(__uint_as_float(a << 16) * g.x, __uint_as_float(b << 16) * g.y);
          }
        }
        if (c % kPer == 0) take(n8, c / kPer);
        if (!ok) break;
        if (works) tc::TmemIo<32>::store(t_op + c * 32, w);
        if (c % kPer == kPer - 1) give(c / kPer);
      }
    }
  } else {
    // ------------------------------------------------------ Q, tree, softmax
    const int cg = warp >> 2;                  // column group
    const int key = (warp & 3) * 32 + lane;
    bool ok = true;
    // Q scaled so that the tile's largest magnitude is in [2^14, 2^15), or each
    // row's own. D / 8 lanes hold a row. A row that is not finite counts for
    // nothing and becomes NaN throughout: all of its scores are NaN then, also
    // where each would be -inf.
    // (The rows' magnitudes lie where the columns' maxima will: those are
    // written once the first product is there, which waits for all of Q.)
    uint32_t* s_qrow = reinterpret_cast<uint32_t*>(s_red[0]);
    uint32_t qmax = 0, qmin = kNotFinite;
#pragma unroll
    for (int k = 0; k < kQSteps; ++k) {
      const uint32_t in[4] = {qv[k].x, qv[k].y, qv[k].z, qv[k].w};
      uint32_t m = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) m = __vmaxu2(m, in[e] & 0x7FFF7FFFu);
      m = max(m & 0xFFFFu, m >> 16);
      if (m >= 0x7F80u) m = kNotFinite;
#pragma unroll
      for (int o = D / 16; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
      const int r = (tid + k * (SW * 32)) / (D / 8);
      if (lane % (D / 8) == 0 && r < R) s_qrow[r] = m;
      if (m < kNotFinite) {
        qmax = max(qmax, m);
        if (m > 0) qmin = min(qmin, m);
      }
    }
    qmax = __reduce_max_sync(0xFFFFFFFFu, qmax);
    qmin = __reduce_min_sync(0xFFFFFFFFu, qmin);
    if (lane == 0) {
      atomicMax(&s_qmax, qmax);
      atomicMin(&s_qmin, qmin);
    }
    if (tid < R) {
      s_neg[tid] = kNoRef;
      s_lo[tid] = 0.0f;
    }
    named_sync(4, SW * 32);
    auto exponent = [](uint32_t m) { return max(static_cast<int>(m >> 7), 20); };
    const int qe = exponent(s_qmax);
    // Beyond 2^73 a zero score would meet an infinite factor of its key's.
    const bool rows_apart = exponent(s_qmin) + kSpread < qe || qe > 200;
    // wide: row r's scores carry 2^(its exponent - qe + lift), keys 2^(qe - lift)
    const int lift = rows_apart ? min(max(qe - 141, 0), 60) : 0;
    if (key < HC) {
      const int e = exponent(s_qrow[cg * HC + key] & 0x7FFFu);
      s_cf[cg * HC + key] = rows_apart ? pow2i(max(e - qe + lift, -126)) : 1.0f;
    }
#pragma unroll
    for (int k = 0; k < kQSteps; ++k) {
      const int it = tid + k * (SW * 32), r = it / (D / 8), j = it % (D / 8);
      if (r < R) {
        const uint32_t m = s_qrow[r];
        const float qf = m >= kNotFinite ? NAN : pow2i(141 - (rows_apart ? exponent(m) : qe));
        *reinterpret_cast<uint4*>(sQ + tc::sw128_offset(r, j, R)) =
            make_uint4(scaled_half2(qv[k].x, qf), scaled_half2(qv[k].y, qf),
                       scaled_half2(qv[k].z, qf), scaled_half2(qv[k].w, qf));
      }
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&b_q);
    // Columns: what each row sees of the tree, and its depth. Only a unit with
    // the tree, or one at the window's edge (whatever the depths), needs it.
    int lo_all = INT32_MIN;   // (no window, or none that reaches this unit)
    if (has_tree || (p.window > 0 && (fb + 2 * c0) * kBlk < C + p.n_nodes - p.window)) {
      if (tid < n_rows) {
        const int grp = tid / HC;
        const uint32_t bit = 1u << (tid - grp * HC);
        int depth = -1;
        for (int x = p.group == 1 ? row0 + tid : static_cast<int>(__umulhi(row0 + tid, p.group_m));
             x >= 0; x = s_parent[x]) {
          atomicOr(&s_see[x][grp], bit);
          ++depth;
        }
        if (depth > p.max_depth) report(p.status, DFV_DEV_DEPTH);
        atomicOr(&s_dep[depth][grp], bit);
        atomicMax(&s_maxdepth, depth);
      }
      named_sync(4, SW * 32);
      const int maxdepth = s_maxdepth;
      for (int k = tid; k < NG * (maxdepth + 1); k += SW * 32) {
        uint32_t m = 0;
        for (int x = 0; x <= k / NG; ++x) m |= s_dep[x][k % NG];
        s_upto[k / NG][k % NG] = m;
      }
      named_sync(4, SW * 32);
      if (p.window > 0) lo_all = C + maxdepth - p.window + 1;
    }
    const float sc = p.scale * kLog2eF * pow2i(qe - 141 - lift);
    float l[HC];
#pragma unroll
    for (int c = 0; c < HC; ++c) l[c] = 0.0f;
    const uint32_t t_s = tmem + lanes + A::kTS + cg * HC;
    const uint32_t t_o = t_s + (A::kTO - A::kTS);
    const float4* m4 = reinterpret_cast<const float4*>(s_neg + cg * HC);
    const float4* lo4 = reinterpret_cast<const float4*>(s_lo + cg * HC);
    const float4* cf4 = reinterpret_cast<const float4*>(s_cf + cg * HC);

    // Chunks [m_lo, m_hi) need no mask: their blocks are complete and inside
    // every node's window. The loop keeps little beside x and l: what a masked
    // chunk needs is worked out in its branch.
    int m_lo = lo_all > 0 ? (lo_all + kBlk - 1) / kBlk - fb - 2 * c0 : 0;   // in blocks, from c0
    m_lo = m_lo > 0 ? (m_lo + 1) / 2 : 0;
    const int m_hi = n8 - (n8 > 0 && fb + 2 * (c0 + n8) > open ? 1 : 0);
    if (n8 > 0) ok = role_wait(&b_sc, 0, &s_dead);

    // Chunks [i0, n), of which the first gets new references; returns the first
    // one not done: n, but for the narrow form where a reference is far out.
    // Wide units have a form of their own, and new references are made beside
    // the loop's common path, not by further turns through it (23 nodes at ctx
    // 131072: 98.2 us; one form with the difference behind a branch 105 to 108,
    // two with three turns a chunk 104.5; narrow alone, in turns, 101.5). A wide
    // tile of 69 rows takes 221 us; unrolled like the narrow form 120, but the
    // narrow one then 100.3, and up to 8 % more at other shapes.
    auto chunks = [&](auto form, const int i0) {
      constexpr bool kWide = decltype(form)::value;
      for (int i = i0; i < n; ++i) {
        // this lane's key: its factors, and the columns that see it
        const bool bf = has_tree && i == n - 1;
        const bool masked = i < m_lo || i >= m_hi;
        uint32_t vis = ~0u;
        bool bad = false, live = true;
        if (masked) {
          const int pos = bf ? open * kBlk + key : (fb + 2 * (c0 + i)) * kBlk + key;
          live = bf ? key < live_rows : pos < open * kBlk;
          if (!live) {
            vis = 0;
          } else if (bf && key >= T) {
            vis = s_see[key - T][cg];
          } else if (lo_all != INT32_MIN) {
            const int dd = pos - C + p.window - 1;   // deepest node that sees it
            vis = dd < 0 ? 0u : s_upto[min(dd, s_maxdepth)][cg];
          }
        }
        ok = ok && role_wait(&b_kfree[A::kKSub - 1], i & 1, &s_dead);
        const float4 scales = s_sc[(i & 31) * 2 + (key >> 6)];
        float a = live ? scales.x * sc : 0.0f, lv = live ? scales.y : 0.0f;
        float iv = live ? scales.z : 0.0f;
        if (bf) {
          ok = ok && role_wait(&b_rowsc, 0, &s_dead);
          if (ok && key < live_rows) {
            a = s_ksc[key] * sc;
            lv = static_cast<float>(s_vexp[key]);
            iv = pow2i(-s_vexp[key]);
            bad = s_bad[0][key] || s_bad[1][key];
          }
        }
        ok = __all_sync(0xFFFFFFFFu, ok);   // the TMEM loads are warp-wide
        tc::fence_after_sync();
        float x[HC];
        // Exponents against the references. Where one is too large, and in the
        // first chunk: scores alone, columns' maxima, new references, and the
        // exponents again. In a wide unit the scores have their column's factor,
        // the key's V scale is added behind the fma, which is exact near the
        // reference, and a second part of the reference takes what rounding has
        // left of the first.
        // kRef 0: no references, 1: both parts, 2: the first part alone
        auto exponents = [&](auto with_ref) {
          constexpr int kRef = decltype(with_ref)::value;
          if (ok) tc::TmemIo<HC>::load(t_s, reinterpret_cast<uint32_t*>(x));
          if constexpr (kWide) {
            // by way of local memory, four columns a turn: the registers are the
            // narrow form's
            float4 xw[HC / 4];
#pragma unroll
            for (int j = 0; j < HC / 4; ++j)
              xw[j] = make_float4(x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]);
#pragma unroll 1
            for (int j = 0; j < HC / 4; ++j) {
              const float4 f = cf4[j];
              float4 y = xw[j], m = make_float4(0.0f, 0.0f, 0.0f, 0.0f), m2 = m;
              if constexpr (kRef != 0) m = m4[j];
              if constexpr (kRef == 1) m2 = lo4[j];
              y.x = fmaf(y.x * f.x, a, m.x) + (lv + m2.x);
              y.y = fmaf(y.y * f.y, a, m.y) + (lv + m2.y);
              y.z = fmaf(y.z * f.z, a, m.z) + (lv + m2.z);
              y.w = fmaf(y.w * f.w, a, m.w) + (lv + m2.w);
              xw[j] = y;
            }
#pragma unroll
            for (int j = 0; j < HC / 4; ++j) {
              x[4 * j] = xw[j].x;
              x[4 * j + 1] = xw[j].y;
              x[4 * j + 2] = xw[j].z;
              x[4 * j + 3] = xw[j].w;
            }
          } else if constexpr (kRef == 0) {
#pragma unroll
            for (int c = 0; c < HC; c += 2) fma2(x[c], x[c + 1], x[c], x[c + 1], a, a, lv, lv);
          } else {
#pragma unroll
            for (int c = 0; c < HC; c += 4) {
              float4 m = m4[c / 4];
              add2(m.x, m.y, m.x, m.y, lv, lv);
              add2(m.z, m.w, m.z, m.w, lv, lv);
              fma2(x[c], x[c + 1], x[c], x[c + 1], a, a, m.x, m.y);
              fma2(x[c + 2], x[c + 3], x[c + 2], x[c + 3], a, a, m.z, m.w);
            }
          }
          if (masked) {
#pragma unroll
            for (int c = 0; c < HC; ++c)
              if (!(vis & (1u << c))) x[c] = -INFINITY;
          }
        };
        auto maxima = [&]() {   // of the columns, by lane; for the group's first warp
#pragma unroll
          for (int c = 0; c < HC; ++c) {
            float m;
            asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(x[c]));
            if (lane == 0) s_red[warp & 3][cg * HC + c] = m;
          }
          named_sync(5 + cg, 128);
          static_assert(HC <= 32, "a lane has one column of the group");
          const int c = cg * HC + min(lane, HC - 1);
          return fmaxf(fmaxf(s_red[0][c], s_red[1][c]), fmaxf(s_red[2][c], s_red[3][c]));
        };
        bool renew = i == i0;
        float top = -INFINITY;
        if (!renew) {
          exponents(std::integral_constant<int, 1>{});
#pragma unroll
          for (int c = 0; c < HC; c += 2) top = max3(top, x[c], x[c + 1]);
          renew = !named_sync_and(5 + cg, 128, ok && !(top > kRaise));
        }
        if (renew) {
          ok = named_sync_and(5 + cg, 128, ok);   // or has a wait given up?
          if (!ok) break;
          const int c = cg * HC + min(lane, HC - 1);
          const bool mine = (warp & 3) == 0 && lane < HC;
          exponents(std::integral_constant<int, 0>{});
          top = maxima();
          float was = -s_neg[c], lo = s_lo[c];
          bool up = top - kTop > was - lo;   // (not with NaN, where the comparison fails)
          if constexpr (!kWide) {
            const bool far = __any_sync(0xFFFFFFFFu, fabsf(top) > kFar && fabsf(top) < INFINITY);
            if (far) return i;   // nothing changes before the wide form
          }
          __syncwarp();
          if (mine && up) s_neg[c] = kTop - top;
          float f = up ? tc::ex2(was - (top - kTop)) : 1.0f;
          if constexpr (kWide) {
            named_sync(5 + cg, 128);
            exponents(std::integral_constant<int, 2>{});
            const float first = top - kTop;
            top = maxima();
            up = up && top > -INFINITY;
            if (mine && up) s_lo[c] = kTop - top;
            f = up ? tc::ex2((was - first) + (kTop - top - lo)) : 1.0f;
          }
          if (mine) s_f[c] = f;
          if (i > 0) ok = role_wait(&b_pv[(i - 1) & 1], ((i - 1) >> 1) & 1, &s_dead);
          ok = named_sync_and(5 + cg, 128, ok);
          if (!ok) break;
          if (i > 0) {
            tc::fence_after_sync();
#pragma unroll
            for (int c = 0; c < HC; ++c) l[c] *= s_f[cg * HC + c];
#pragma unroll 1
            for (int hh = 0; hh < A::kHalves; ++hh) {
              tc::TmemIo<HC>::load(t_o + hh * R, reinterpret_cast<uint32_t*>(x));
#pragma unroll
              for (int c = 0; c < HC; ++c) x[c] *= s_f[cg * HC + c];
              tc::TmemIo<HC>::store(t_o + hh * R, reinterpret_cast<const uint32_t*>(x));
              tc::store_wait();
            }
          }
          exponents(std::integral_constant<int, 1>{});
        }
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&b_sfree);
        if (bad) {   // whoever sees the key has no result
#pragma unroll
          for (int c = 0; c < HC; ++c) {
            if (x[c] > -INFINITY) l[c] = NAN;
            x[c] = -INFINITY;
          }
        }
        // P' as the B operand: 16-byte pieces of 8 columns of this key's row
        const int pb = i & 1;
        if (A::kPBufs == 1 && i >= 1) ok = role_wait(&b_pv[pb ^ 1], ((i - 1) >> 1) & 1, &s_dead);
        if (ok) {
          uint8_t* dst = sP + (A::kPBufs == 2 ? pb : 0) * A::kPBytes;
          const uint32_t krow = static_cast<uint32_t>((key >> 3) * 1024 + (key & 7) * 128);
#pragma unroll
          for (int j = 0; j < HC / 4; ++j) {   // half a 16-byte piece
            uint32_t o[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int c = 4 * j + 2 * e;
              const float p0 = tc::ex2(x[c]), p1 = tc::ex2(x[c + 1]);
              fma2(l[c], l[c + 1], p0, p1, iv, iv, l[c], l[c + 1]);
              o[e] = pack_half2(p0, p1);
            }
            const int col = cg * HC + 4 * j, piece = col >> 3;
            *reinterpret_cast<uint2*>(dst + (piece >> 3) * (kAtKeys * 128) + krow +
                                      (((piece & 7) ^ (key & 7)) << 4) + (col & 4) * 2) =
                make_uint2(o[0], o[1]);
          }
        }
        fence_proxy_async_smem();
        if (__all_sync(0xFFFFFFFFu, ok) && lane == 0) mbar_arrive(&b_p[pb]);
      }
      return n;
    };
    const int done = rows_apart ? 0 : chunks(std::false_type{}, 0);
    if (done < n) chunks(std::true_type{}, done);
    // ---- the unit's result
    // sums over the lanes, four columns at a time: two exchanges that halve
    // the columns a lane holds, then three plain ones
#pragma unroll
    for (int c = 0; c < HC; c += 4) {
      float s2[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float send = lane & 16 ? l[c + k] : l[c + 2 + k];
        s2[k] = (lane & 16 ? l[c + 2 + k] : l[c + k]) + __shfl_xor_sync(0xFFFFFFFFu, send, 16);
      }
      const float send = lane & 8 ? s2[0] : s2[1];
      float s = (lane & 8 ? s2[1] : s2[0]) + __shfl_xor_sync(0xFFFFFFFFu, send, 8);
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
      if ((lane & 7) == 0) s_red[warp & 3][cg * HC + c + (lane >> 4) * 2 + ((lane >> 3) & 1)] = s;
    }
    named_sync(5 + cg, 128);
    const int64_t slice = (static_cast<int64_t>(h) * gridDim.y + tile) * splits + split;
    if ((warp & 3) == 0) {
      for (int c = cg * HC + lane; c < (cg + 1) * HC; c += 32) {
        const float s = (s_red[0][c] + s_red[1][c]) + (s_red[2][c] + s_red[3][c]);
        s_f[c] = s == 0.0f ? 0.0f : 1.0f / s;
        p.part_lse[slice * R + c] = s == 0.0f ? -INFINITY : (log2f(s) - s_lo[c]) - s_neg[c];
      }
    }
    if (ok && n > 0) ok = role_wait(&b_pv[(n - 1) & 1], ((n - 1) >> 1) & 1, &s_dead);
    ok = named_sync_and(5 + cg, 128, ok);
    if (ok && n > 0) {
      tc::fence_after_sync();
      float* dst = p.part_o + (slice * R + cg * HC) * D + key;
      const float4* f4 = reinterpret_cast<const float4*>(s_f + cg * HC);
#pragma unroll 1
      for (int hh = 0; hh < A::kHalves; ++hh) {
        float x[HC];
        tc::TmemIo<HC>::load(t_o + hh * R, reinterpret_cast<uint32_t*>(x));
        if (D >= 128 || key < D) {
#pragma unroll
          for (int c = 0; c < HC; c += 4) {
            if (cg * HC + c >= n_rows) break;   // rows past the tile's
            const float4 f = f4[c / 4];
            dst[hh * 128 + c * D] = x[c] * f.x;
            dst[hh * 128 + (c + 1) * D] = x[c + 1] * f.y;
            dst[hh * 128 + (c + 2) * D] = x[c + 2] * f.z;
            dst[hh * 128 + (c + 3) * D] = x[c + 3] * f.w;
          }
        }
      }
    }
    tc::fence_before_sync();
  }
  __syncwarp();
  __syncthreads();
  if (warp == SW + 8) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, 512);
  }
  if (tid == 0 && s_dead) report(p.status, DFV_DEV_TIMEOUT);
}

// Slices of the keys joined: one CTA per (node, query head) row weighs the
// partial rows by 2^(lse - largest lse) in a fixed order. Latency bound; the
// launch overlaps the attention's end.
constexpr int kMergeThreads = 128;
constexpr int kMaxSplits = 256;

struct MergeParams {
  int splits, r, tiles, rows_tile, hq, group;
  const float* part_o;
  const float* part_lse;
  void* out;
  int out_bf16;
  float* lse;
};

template <int D>
__global__ void __launch_bounds__(kMergeThreads)
    kv8_merge_kernel(const __grid_constant__ MergeParams p) {
  constexpr int kV = D / 4, kG = kMergeThreads / kV;   // float4 of a row; groups of splits
  __shared__ float s_w[kMaxSplits];
  __shared__ float4 s_o[kG][kV];
  const int tid = threadIdx.x, lane = tid & 31, splits = p.splits;
  const int head = blockIdx.x, node = blockIdx.y;
  const int h = head / p.group, r = node * p.group + head - h * p.group;
  const int tile = r / p.rows_tile;
  const int64_t row = static_cast<int64_t>(node) * p.hq + head;
  // this row of slice 0, and what lies between slices
  const int64_t at = ((static_cast<int64_t>(h) * p.tiles + tile) * splits) * p.r + r -
                     tile * p.rows_tile;
  const float* part_lse = p.part_lse + at;
  const float* part_o = p.part_o + at * D;
  // The attention has triggered behind its wait, so what ran before the call
  // has completed; what follows may be set up under the attention itself.
  grid_dep_launch_dependents();
  grid_dep_wait();
  float m = -INFINITY;
  for (int s = lane; s < splits; s += 32) m = fmaxf(m, part_lse[s * p.r]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  float total = 0.0f;
  for (int s = lane; s < splits; s += 32) {
    const float v = part_lse[s * p.r];
    const float w = v == -INFINITY ? 0.0f : tc::ex2(v - m);
    total += w;
    if (tid < 32) s_w[s] = w;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xFFFFFFFFu, total, o);
  __syncthreads();
  float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
  for (int s = tid / kV; s < splits; s += kG) {
    const float w = s_w[s];
    if (w == 0.0f) continue;   // an empty slice has no row
    const float4 v =
        reinterpret_cast<const float4*>(part_o + static_cast<int64_t>(s) * p.r * D)[tid % kV];
    a.x = fmaf(w, v.x, a.x);
    a.y = fmaf(w, v.y, a.y);
    a.z = fmaf(w, v.z, a.z);
    a.w = fmaf(w, v.w, a.w);
  }
  s_o[tid / kV][tid % kV] = a;
  __syncthreads();
  if (tid < kV) {
#pragma unroll
    for (int g = 1; g < kG; ++g) {
      a.x += s_o[g][tid].x;
      a.y += s_o[g][tid].y;
      a.z += s_o[g][tid].z;
      a.w += s_o[g][tid].w;
    }
    const float inv = total == 0.0f ? 0.0f : 1.0f / total;
    a.x *= inv;
    a.y *= inv;
    a.z *= inv;
    a.w *= inv;
    if (p.out_bf16) {
      const __nv_bfloat162 lo = __floats2bfloat162_rn(a.x, a.y);
      const __nv_bfloat162 hi = __floats2bfloat162_rn(a.z, a.w);
      reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + row * D)[tid] =
          make_uint2(*reinterpret_cast<const uint32_t*>(&lo),
                     *reinterpret_cast<const uint32_t*>(&hi));
    } else {
      reinterpret_cast<float4*>(static_cast<float*>(p.out) + row * D)[tid] = a;
    }
  }
  if (tid == 0 && p.lse)
    p.lse[row] = total == 0.0f ? -INFINITY : (m + log2f(total)) * kLn2F;
}

// ---------------------------------------------------------------- host

struct AttnPlan {
  int tiles, rows_tile, r, splits;
};

// Query rows of a tile: TMEM columns bound it at D = 256, the softmax's
// registers (a quarter of the columns a thread, twice) below.
constexpr int max_rows(int d) { return d == 256 ? 80 : 96; }

// The fewest tiles, as even as they come. Slices: the SMs take units in waves,
// a unit costs its chunks plus its start and end, and each slice adds its
// partial rows, written and read once. Measured at ctx 61440, window 2048, 23
// nodes (18 chunks, 8 units, 0.28 us of partial rows a slice): 6, 9, 12 and
// 18 slices take 20.4, 16.2, 18.2 and 17.7 us; the model says 9.
static AttnPlan attn_plan(int n_nodes, int hq, int hkv, int d, int window, int capacity) {
  AttnPlan pl;
  const int rows = n_nodes * (hq / hkv);
  pl.tiles = (rows + max_rows(d) - 1) / max_rows(d);
  pl.rows_tile = (rows + pl.tiles - 1) / pl.tiles;
  pl.r = (pl.rows_tile + 15) / 16 * 16;
  const int span = window > 0 && window < capacity ? window : capacity;
  const int chunks = span / kAtKeys + 2;
  const int64_t units = static_cast<int64_t>(hkv) * pl.tiles;
  const int sms = sm_count();
  const int most = chunks < kMaxSplits ? chunks : kMaxSplits;
  const double chunk_us = 0.4 + d / 256.0 * (1.0 + 0.6 * pl.r / 80.0);
  const double merge_us = static_cast<double>(n_nodes) * hq * d * 8 / 4e6;   // of one slice
  double best = 1e30;
  pl.splits = 1;
  for (int s = 1; s <= most && (s == 1 || units * s <= 4 * sms); ++s) {
    const double cost = ((units * s + sms - 1) / sms) * ((chunks + s - 1) / s * chunk_us + 6.0) +
                        s * merge_us;
    if (cost < best) {
      best = cost;
      pl.splits = s;
    }
  }
  return pl;
}

static bool attn_shape_ok(int n_nodes, int hq, int hkv, int d, int window, int capacity) {
  return n_nodes >= 1 && n_nodes <= kMaxNodes && hkv >= 1 && hq >= 1 && hq % hkv == 0 &&
         hq <= 256 && kv8_dim_ok(d) && window >= 0 && capacity >= 1 && capacity <= (1 << 30);
}

static size_t attn_ws_bytes(const AttnPlan& pl, int hkv, int d) {
  return static_cast<size_t>(hkv) * pl.tiles * pl.splits * pl.r * (d + 1) * sizeof(float);
}

template <int D, int R>
static dfv_status attn_launch(const AttnParams& p, const MergeParams& m, cudaStream_t stream) {
  using A = AttnShape<D, R>;
  static std::atomic<int> configured[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return DFV_ERR_CUDA;
  if (!configured[dev].load(std::memory_order_acquire)) {
    if (cudaFuncSetAttribute(kv8_attn_kernel<D, R>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             A::kBytes) != cudaSuccess)
      return DFV_ERR_CUDA;
    configured[dev].store(1, std::memory_order_release);
  }
  // both launches may be set up while the kernel before them runs
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(m.splits, m.tiles, p.c.n_kv_heads);
  cfg.blockDim = dim3(A::kThreads);
  cfg.dynamicSmemBytes = A::kBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kv8_attn_kernel<D, R>, p) != cudaSuccess) return DFV_ERR_CUDA;
  cfg.gridDim = dim3(p.hq, p.n_nodes);
  cfg.blockDim = dim3(kMergeThreads);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, kv8_merge_kernel<D>, m) == cudaSuccess ? DFV_OK : DFV_ERR_CUDA;
}

template <int D>
static dfv_status attn_launch_r(const AttnParams& p, const MergeParams& m, cudaStream_t stream) {
  switch (m.r) {
    case 16: return attn_launch<D, 16>(p, m, stream);
    case 32: return attn_launch<D, 32>(p, m, stream);
    case 48: return attn_launch<D, 48>(p, m, stream);
    case 64: return attn_launch<D, 64>(p, m, stream);
    case 80: return attn_launch<D, 80>(p, m, stream);
    default:
      if constexpr (D <= 128) return attn_launch<D, 96>(p, m, stream);
      return DFV_ERR_UNSUPPORTED;
  }
}

}  // namespace dfv

extern "C" size_t dfv_kv8_attn_workspace_bytes(int n_nodes, int n_q_heads, int n_kv_heads,
                                               int head_dim, int window, int cache_capacity) {
  using namespace dfv;
  if (!attn_shape_ok(n_nodes, n_q_heads, n_kv_heads, head_dim, window, cache_capacity)) return 0;
  return attn_ws_bytes(attn_plan(n_nodes, n_q_heads, n_kv_heads, head_dim, window, cache_capacity),
                       n_kv_heads, head_dim);
}

extern "C" dfv_status dfv_kv8_attn(const dfv_kv8_cache* cache, int n_nodes, int max_depth,
                                   int n_q_heads, int window, const void* q, const void* tree_k,
                                   const void* tree_v, const int32_t* parent, float scale,
                                   void* out, int out_dtype, float* lse, void* workspace,
                                   size_t workspace_bytes, uint32_t* status, dfv_stream_t stream) {
  using namespace dfv;
  if (!kv8_cache_ok(cache)) return DFV_ERR_INVALID;
  const int hkv = cache->n_kv_heads, d = cache->head_dim;
  if (!kv8_dim_ok(d) || (out_dtype != DFV_DTYPE_F32 && out_dtype != DFV_DTYPE_BF16))
    return DFV_ERR_UNSUPPORTED;
  if (!attn_shape_ok(n_nodes, n_q_heads, hkv, d, window, cache->capacity) || max_depth < 0)
    return DFV_ERR_INVALID;
  if (!q || !tree_k || !tree_v || !parent || !out || !aligned(q, 16) || !aligned(tree_k, 16) ||
      !aligned(tree_v, 16) || !aligned(out, 16))
    return DFV_ERR_INVALID;
  const AttnPlan pl = attn_plan(n_nodes, n_q_heads, hkv, d, window, cache->capacity);
  if (!workspace || !aligned(workspace, 256)) return DFV_ERR_INVALID;
  if (workspace_bytes < attn_ws_bytes(pl, hkv, d)) return DFV_ERR_WORKSPACE;
  AttnParams p = {};
  p.c = *cache;
  p.nblk = kv8_blocks(cache->capacity);
  p.n_nodes = n_nodes;
  p.max_depth = max_depth;
  p.hq = n_q_heads;
  p.group = n_q_heads / hkv;
  p.window = window;
  p.group_m = static_cast<uint32_t>(((1ull << 32) + p.group - 1) / p.group);   // exact below 2^24
  p.rows = n_nodes * p.group;
  p.rows_tile = pl.rows_tile;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.tree_k = static_cast<const __nv_bfloat16*>(tree_k);
  p.tree_v = static_cast<const __nv_bfloat16*>(tree_v);
  p.parent = parent;
  p.scale = scale > 0.0f ? scale : 1.0f / sqrtf(static_cast<float>(d));
  p.part_o = static_cast<float*>(workspace);
  p.part_lse = p.part_o + static_cast<size_t>(hkv) * pl.tiles * pl.splits * pl.r * d;
  p.status = status;
  const MergeParams m = {pl.splits, pl.r, pl.tiles, pl.rows_tile, n_q_heads, p.group, p.part_o,
                         p.part_lse, out, out_dtype == DFV_DTYPE_BF16, lse};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  switch (d) {
    case 64: return attn_launch_r<64>(p, m, s);
    case 128: return attn_launch_r<128>(p, m, s);
    default: return attn_launch_r<256>(p, m, s);
  }
}
