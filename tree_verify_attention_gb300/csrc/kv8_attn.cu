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
// to show that no exponent passes 2^10 (binary16 P' holds 2^15), which one
// vote decides; columns' maxima are reduced across lanes only when one does.
// The tail and tree rows (bf16) are one last chunk of at most 63 + 65 = 128
// keys, scaled by a power of two per key to binary16 range, so that it runs
// through the same products with its own a_j and v_scale_j. Q is scaled by one
// power of two per tile. Every operand is then exact in binary16 except P',
// whose rounding (2^-12) is below that of the bf16 output.
//
// Roles of a CTA (one per SM): warps 0-7 softmax (lane quadrant w % 4, column
// half w / 4), warps 8-11 K codes to TMEM, warps 12-15 V codes, warp 16 issues
// MMAs, warp 17 bulk copies. A unit is (KV head, tile of at most 80 query
// rows, slice of the chunks). Bound by HBM while a tile has few rows, by the
// softmax and the decode for many.

#include <atomic>
#include <math.h>

#include "kv8.cuh"
#include "tc.cuh"
#include "tmem_io.cuh"

namespace dfv {

constexpr int kAtThreads = 576;
constexpr int kAtKeys = 128;         // keys of a chunk
constexpr float kRaise = 10.0f;      // a larger exponent moves the reference
constexpr float kNoRef = -1e30f;     // reference of a column that has seen no key
constexpr float kLog2eF = 1.4426950408889634f;
constexpr float kLn2F = 0.6931471805599453f;

template <int D, int R>
struct AttnShape {
  static constexpr int kHalves = D == 256 ? 2 : 1;      // 128-lane parts of V^T
  static constexpr int kRaw = kAtKeys * D;              // bytes of a chunk's K (V) codes
  static constexpr int kPBlk = (R + 63) / 64;
  static constexpr int kPBytes = kPBlk * kAtKeys * 128;
  static constexpr int kPBufs = R <= 64 || D < 256 ? 2 : 1;
  static constexpr int kStages = D == 256 ? 2 : 4;
  static constexpr int kQBytes = R * D * 2;
  static constexpr int kOffQ = kStages * 2 * kRaw;
  static constexpr int kOffP = (kOffQ + kQBytes + 1023) / 1024 * 1024;
  static constexpr int kBytes = kOffP + kPBufs * kPBytes + 1024;
  // TMEM columns
  static constexpr uint32_t kTK = 0;
  static constexpr uint32_t kTV = kTK + D / 2;
  static constexpr uint32_t kTS = kTV + 64 * kHalves;
  static constexpr uint32_t kTO = kTS + R;
  static_assert(kTO + R * kHalves <= 512, "TMEM columns");
  static_assert(kBytes <= 227 * 1024, "shared memory");
};

struct AttnParams {
  dfv_kv8_cache c;
  int nblk;
  int n_nodes, max_depth, hq, group, window;
  int tiles, rows_tile, rows, splits;   // rows: of one KV head
  const __nv_bfloat16* q;
  const __nv_bfloat16* tree_k;
  const __nv_bfloat16* tree_v;
  const int32_t* parent;
  float scale;
  void* out;
  int out_bf16;
  float* lse;
  float* part_o;     // [split][node][query head][D], normalised (splits > 1)
  float* part_lse;   // [split][node][query head], base 2
  uint32_t* status;
};

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// Bounded wait that also gives up when another role has.
__device__ __forceinline__ bool role_wait(uint64_t* bar, uint32_t parity, volatile int* dead) {
  if (mbar_try_wait(bar, parity)) return true;
  bool there = false;
  const bool ended = wait_bounded([&]() {
    there = mbar_try_wait(bar, parity);
    return there || *dead;
  });
  if (!ended) *dead = 1;
  return there;
}

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

__device__ __forceinline__ float pow2i(int e) {   // e in [-126, 127]
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// Byte offset of the 16-byte piece j (8 dims) of key k in a staged bf16-chunk
// operand: consecutive keys are adjacent, and the exclusive or keeps both a
// row's pieces and a dim's keys off one another's banks.
__device__ __forceinline__ int stage_piece(int j, int k) {
  return (j * kAtKeys + (k ^ (j & 7))) * 16;
}

template <int D, int R>
__global__ void __launch_bounds__(kAtThreads, 1)
    kv8_attn_kernel(const __grid_constant__ AttnParams p) {
  using A = AttnShape<D, R>;
  constexpr int HC = R / 2;   // columns of a softmax thread
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* sQ = smem + A::kOffQ;
  uint8_t* sP = smem + A::kOffP;
  __shared__ uint64_t b_kfull[4], b_kfree[4], b_vfull[4], b_vfree[4];
  __shared__ uint64_t b_khat, b_vhat, b_sfull, b_sfree, b_q, b_end, b_p[2], b_pv[2];
  __shared__ uint32_t s_tmem;
  __shared__ volatile int s_dead;
  __shared__ int s_parent[kMaxNodes], s_maxdepth;
  __shared__ uint32_t s_anc[kMaskWords][R];
  __shared__ int s_lo[R], s_row[R];   // first visible position; row of the output
  __shared__ __align__(16) float s_m[R], s_f[R];
  __shared__ float s_red[4][R];
  __shared__ float s_ksc[kAtKeys];
  __shared__ int s_vexp[kAtKeys];
  __shared__ int s_badk[kAtKeys], s_badv[kAtKeys];
  __shared__ uint32_t s_qmax;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  grid_dep_launch_dependents();   // the merge may be set up meanwhile
  const int split = blockIdx.x % p.splits, unit = blockIdx.x / p.splits;
  const int tile = unit % p.tiles, h = unit / p.tiles;
  const int row0 = tile * p.rows_tile, n_rows = min(p.rows_tile, p.rows - row0);
  int C = *p.c.state;
  if (C < 0 || C > p.c.capacity) {
    if (tid == 0) report(p.status, DFV_DEV_CTX);
    C = max(0, min(C, p.c.capacity));
  }
  // chunks: complete blocks [fb, open) two at a time, then the bf16 chunk
  const int open = C / kBlk, T = C % kBlk;
  const int lo_min = p.window > 0 ? max(0, C - p.window + 1) : 0;
  const int fb = min(lo_min / kBlk, open);
  const int nq = (open - fb + 1) / 2, nch = nq + 1;
  const int c0 = static_cast<int>(static_cast<int64_t>(nch) * split / p.splits);
  const int c1 = static_cast<int>(static_cast<int64_t>(nch) * (split + 1) / p.splits);
  const int n = c1 - c0;
  const bool has_tree = c1 == nch && n > 0;     // its last chunk is the bf16 one
  const int n8 = n - (has_tree ? 1 : 0);

  if (tid == 0) {
    s_dead = 0;
    s_qmax = 0;
    s_maxdepth = 0;
    for (int s = 0; s < A::kStages; ++s) {
      mbar_init(&b_kfull[s], 1);
      mbar_init(&b_vfull[s], 1);
      mbar_init(&b_kfree[s], 4);
      mbar_init(&b_vfree[s], 4);
    }
    mbar_init(&b_khat, 4);
    mbar_init(&b_vhat, 4);
    mbar_init(&b_sfull, 1);
    mbar_init(&b_sfree, 8);
    mbar_init(&b_q, 8);
    mbar_init(&b_end, 1);
    for (int k = 0; k < 2; ++k) {
      mbar_init(&b_p[k], 8);
      mbar_init(&b_pv[k], 1);
    }
    fence_mbar_init();
  }
  if (warp == 16) tc::tmem_alloc(&s_tmem, 512);
  for (int i = tid; i < p.n_nodes; i += kAtThreads) {
    int pa = i == 0 ? -1 : p.parent[i];
    if (i > 0 && (pa < 0 || pa >= i)) {
      report(p.status, DFV_DEV_BAD_TREE);
      pa = 0;
    }
    s_parent[i] = pa;
  }
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = s_tmem;
  const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;   // first lane of the quadrant << 16

  if (warp == 17) {
    // ------------------------------------------------------ bulk copies
    if (lane == 0) {
      int issued = 0;
      for (int i = 0; i < n8; ++i) {
        const int s = i % A::kStages, use = i / A::kStages;
        if (use > 0 && (!role_wait(&b_kfree[s], (use - 1) & 1, &s_dead) ||
                        !role_wait(&b_vfree[s], (use - 1) & 1, &s_dead)))
          break;
        const int b = fb + 2 * (c0 + i);
        const uint32_t bytes = static_cast<uint32_t>(min(2, open - b) * kBlk * D);
        const int64_t off = (static_cast<int64_t>(h) * p.nblk + b) * kBlk * D;
        uint8_t* raw = smem + s * 2 * A::kRaw;
        mbar_arrive_expect_tx(&b_kfull[s], bytes);
        bulk_g2s(raw, p.c.k_codes + off, bytes, &b_kfull[s]);
        mbar_arrive_expect_tx(&b_vfull[s], bytes);
        bulk_g2s(raw + A::kRaw, p.c.v_codes + off, bytes, &b_vfull[s]);
        issued = i + 1;
      }
      // copies that nobody will wait for any more must still land
      for (int i = max(0, issued - A::kStages); i < issued; ++i) {
        const uint32_t ph = (i / A::kStages) & 1;
        if (s_dead) {
          mbar_wait_bounded(&b_kfull[i % A::kStages], ph);
          mbar_wait_bounded(&b_vfull[i % A::kStages], ph);
        }
      }
    }
  } else if (warp == 16) {
    // ------------------------------------------------------ MMA issue
    if (lane == 0 && n > 0) {
      constexpr uint32_t id_s = tc::idesc_f16(128, R);
      constexpr uint32_t id_o = tc::idesc_f16(128, R, true);
      const uint64_t qd = tc::smem_desc_sw128(smem_u32(sQ), 1024);
      auto issue_s = [&](int i) {
        if (!role_wait(&b_khat, i & 1, &s_dead)) return false;
        if (i > 0 && !role_wait(&b_sfree, (i - 1) & 1, &s_dead)) return false;
        tc::fence_after_sync();
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          tc::mma_f16_ts(tmem + A::kTS, tmem + A::kTK + kk * 8,
                         qd + static_cast<uint64_t>(((kk >> 2) * R * 128 + (kk & 3) * 32) >> 4),
                         id_s, kk > 0 ? 1u : 0u);
        tc::commit(&b_sfull);
        return true;
      };
      bool ok = role_wait(&b_q, 0, &s_dead) && issue_s(0);
      for (int i = 0; ok && i < n; ++i) {
        if (i + 1 < n) ok = issue_s(i + 1);
        const int pb = i & 1;
        ok = ok && role_wait(&b_vhat, i & 1, &s_dead) &&
             role_wait(&b_p[pb], (i >> 1) & 1, &s_dead);
        if (!ok) break;
        tc::fence_after_sync();
        const uint64_t pd = tc::smem_desc_sw128_mn(
            smem_u32(sP + (A::kPBufs == 2 ? pb : 0) * A::kPBytes), kAtKeys * 128, 1024);
#pragma unroll
        for (int hh = 0; hh < A::kHalves; ++hh)
#pragma unroll
          for (int kk = 0; kk < kAtKeys / 16; ++kk)
            tc::mma_f16_ts(tmem + A::kTO + hh * R, tmem + A::kTV + hh * 64 + kk * 8,
                           pd + static_cast<uint64_t>((kk * 16 * 128) >> 4), id_o,
                           i > 0 || kk > 0 ? 1u : 0u);
        tc::commit(&b_pv[pb]);
      }
      if (!ok) {
        s_dead = 1;
        // MMAs in flight must end before TMEM is freed
        tc::commit(&b_end);
        mbar_wait_bounded(&b_end, 0);
      }
    }
  } else if (warp >= 8) {
    // ------------------------------------------------------ codes to TMEM
    const bool is_v = warp >= 12;
    const int slot = (warp & 3) * 32 + lane;   // key (K) or dim of a half (V)
    uint64_t* full = is_v ? b_vfull : b_kfull;
    uint64_t* free_ = is_v ? b_vfree : b_kfree;
    bool ok = true;
    // the operand's columns are free once the products that read them end
    auto operand_free = [&](int i) {
      if (i == 0) return true;
      return is_v ? role_wait(&b_pv[(i - 1) & 1], ((i - 1) >> 1) & 1, &s_dead)
                  : role_wait(&b_sfull, (i - 1) & 1, &s_dead);
    };
    for (int i = 0; ok && i < n8; ++i) {
      const int s = i % A::kStages;
      const uint8_t* raw = smem + s * 2 * A::kRaw + (is_v ? A::kRaw : 0);
      ok = role_wait(&full[s], (i / A::kStages) & 1, &s_dead) && operand_free(i);
      ok = __all_sync(0xFFFFFFFFu, ok);
      if (!ok) break;
      tc::fence_after_sync();
      if (!is_v) {
        const uint8_t* mine = raw + (slot >> 6) * kBlk * D + (slot & 63) * 16;
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
          uint32_t w[32];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            codes_to_half(*reinterpret_cast<const uint4*>(mine + (c * 4 + j) * kBlk * 16), w + 8 * j);
          tc::TmemIo<32>::store(tmem + lanes + A::kTK + c * 32, w);
        }
      } else if (D >= 128 || slot < D) {   // whole warps
#pragma unroll
        for (int hh = 0; hh < A::kHalves; ++hh)
#pragma unroll
          for (int c = 0; c < 2; ++c) {    // the chunk's blocks
            const uint8_t* mine = raw + c * kBlk * D + (hh * 128 + slot) * 16;
            uint32_t w[32];
#pragma unroll
            for (int j = 0; j < 4; ++j)
              codes_to_half(*reinterpret_cast<const uint4*>(mine + j * D * 16), w + 8 * j);
            tc::TmemIo<32>::store(tmem + lanes + A::kTV + hh * 64 + c * 32, w);
          }
      }
      tc::store_wait();
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&free_[s]);
        mbar_arrive(is_v ? &b_vhat : &b_khat);
      }
    }
    if (has_tree) {
      // The bf16 chunk: key slots [0, T) are the open block's rows, then the
      // tree nodes. Rows are read whole, scaled to binary16 by a power of two
      // (largest magnitude in [64, 128)) and staged over the raw codes, K
      // over the first stage and V over the second.
      ok = named_sync_and(1, 256, ok);   // all earlier codes have been read
      constexpr int LPK = D / 8, KPI = 32 / LPK;   // lanes per key, keys per step
      constexpr int NS = 32 / KPI;                 // steps for the warp's 32 keys
      constexpr int NB = NS < 16 ? NS : 16;        // loads in flight
      uint8_t* stage = smem + (is_v ? 2 * A::kRaw : 0);
      const int j = lane % LPK;
      if (ok) {
#pragma unroll 1
        for (int st = 0; st < NS; st += NB) {
          uint4 v[NB];
#pragma unroll
          for (int u = 0; u < NB; ++u) {
            const int k = (warp & 3) * 32 + (st + u) * KPI + lane / LPK;
            const __nv_bfloat16* src = nullptr;
            if (k < T)
              src = static_cast<const __nv_bfloat16*>(is_v ? p.c.v_tail : p.c.k_tail) +
                    ((static_cast<int64_t>(h) * 2 + (open & 1)) * kBlk + k) * D;
            else if (k < T + p.n_nodes)
              src = (is_v ? p.tree_v : p.tree_k) +
                    (static_cast<int64_t>(k - T) * p.c.n_kv_heads + h) * D;
            v[u] = src ? *reinterpret_cast<const uint4*>(src + j * 8) : make_uint4(0, 0, 0, 0);
          }
#pragma unroll
          for (int u = 0; u < NB; ++u) {
            const int k = (warp & 3) * 32 + (st + u) * KPI + lane / LPK;
            uint32_t in[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
            uint32_t m = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) m = __vmaxu2(m, in[e] & 0x7FFF7FFFu);
            m = max(m & 0xFFFFu, m >> 16);
#pragma unroll
            for (int o = LPK / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
            const bool bad = m >= kBigBits;   // infinite, NaN or out of range
            const int e = max(static_cast<int>(m >> 7), 86);
            const float f = bad ? 0.0f : pow2i(133 - e);
            uint32_t o[4];
#pragma unroll
            for (int q = 0; q < 4; ++q)
              o[q] = bad ? 0u
                         : pack_half2(__uint_as_float(in[q] << 16) * f,
                                      __uint_as_float(in[q] & 0xFFFF0000u) * f);
            *reinterpret_cast<uint4*>(stage + stage_piece(j, k)) = make_uint4(o[0], o[1], o[2], o[3]);
            if (j == 0) {
              if (is_v) {
                s_vexp[k] = bad ? 0 : e - 133;
                s_badv[k] = bad;
              } else {
                s_ksc[k] = bad ? 0.0f : pow2i(e - 133);
                s_badk[k] = bad;
              }
            }
            if (bad && k < T + p.n_nodes && j == 0) report(p.status, DFV_DEV_NONFINITE);
          }
        }
      }
      ok = ok && operand_free(n8);
      ok = named_sync_and(is_v ? 3 : 2, 128, ok);   // this operand's rows are staged
      if (ok) {
        tc::fence_after_sync();
        if (!is_v) {
#pragma unroll
          for (int c = 0; c < D / 64; ++c) {
            uint32_t w[32];
#pragma unroll
            for (int q = 0; q < 8; ++q) {
              const uint4 x = *reinterpret_cast<const uint4*>(stage + stage_piece(c * 8 + q, slot));
              w[4 * q] = x.x;
              w[4 * q + 1] = x.y;
              w[4 * q + 2] = x.z;
              w[4 * q + 3] = x.w;
            }
            tc::TmemIo<32>::store(tmem + lanes + A::kTK + c * 32, w);
          }
        } else if (D >= 128 || slot < D) {
#pragma unroll 1
          for (int hc = 0; hc < 2 * A::kHalves; ++hc) {
            const int d = (hc >> 1) * 128 + slot, kb = (hc & 1) * 64;
            uint32_t w[32];
#pragma unroll
            for (int q = 0; q < 32; ++q) {
              const uint16_t a = *reinterpret_cast<const uint16_t*>(
                  stage + stage_piece(d >> 3, kb + 2 * q) + (d & 7) * 2);
              const uint16_t b = *reinterpret_cast<const uint16_t*>(
                  stage + stage_piece(d >> 3, kb + 2 * q + 1) + (d & 7) * 2);
              w[q] = a | (static_cast<uint32_t>(b) << 16);
            }
            tc::TmemIo<32>::store(tmem + lanes + A::kTV + (hc >> 1) * 64 + (hc & 1) * 32, w);
          }
        }
        tc::store_wait();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(is_v ? &b_vhat : &b_khat);
      }
    }
  } else {
    // ------------------------------------------------------ Q, tree, softmax
    const int cg = warp >> 2;                  // column half
    const int key = (warp & 3) * 32 + lane;
    bool ok = true;
    // Q rows of the tile, scaled so that the largest magnitude is in [2^14, 2^15)
    constexpr int kQSteps = (R * D / 8 + 255) / 256;
    float qs;
    {
      uint4 v[kQSteps];
      uint32_t m = 0;
#pragma unroll
      for (int k = 0; k < kQSteps; ++k) {
        const int it = tid + k * 256, r = it / (D / 8), j = it % (D / 8);
        v[k] = make_uint4(0, 0, 0, 0);
        if (r < n_rows) {
          const int g = (row0 + r) % p.group, node = (row0 + r) / p.group;
          v[k] = *reinterpret_cast<const uint4*>(
              p.q + (static_cast<int64_t>(node) * p.hq + h * p.group + g) * D + j * 8);
        }
        const uint32_t in[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t lo = in[e] & 0x7FFFu, hi = (in[e] >> 16) & 0x7FFFu;
          if (lo < 0x7F80u) m = max(m, lo);   // infinities and NaN stay in their row
          if (hi < 0x7F80u) m = max(m, hi);
        }
      }
      m = __reduce_max_sync(0xFFFFFFFFu, m);
      if (lane == 0) atomicMax(&s_qmax, m);
      named_sync(4, 256);
      const int e = max(static_cast<int>(s_qmax >> 7), 20);
      const float f = pow2i(min(141 - e, 126));
      qs = pow2i(max(e - 141, -126));
#pragma unroll
      for (int k = 0; k < kQSteps; ++k) {
        const int it = tid + k * 256, r = it / (D / 8), j = it % (D / 8);
        if (r >= R) continue;
        const uint32_t in[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
        uint32_t o[4];
#pragma unroll
        for (int q = 0; q < 4; ++q)
          o[q] = pack_half2(__uint_as_float(in[q] << 16) * f,
                            __uint_as_float(in[q] & 0xFFFF0000u) * f);
        *reinterpret_cast<uint4*>(sQ + tc::sw128_offset(r, j, R)) = make_uint4(o[0], o[1], o[2], o[3]);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&b_q);
    }
    // columns: what each row sees of the tree and of the window
    if (tid < R) {
      uint32_t a[kMaskWords] = {};
      int depth = 0, node;
      if (tid < n_rows) {
        node = (row0 + tid) / p.group;
        s_row[tid] = node * p.hq + h * p.group + (row0 + tid) % p.group;
        for (int x = node; x >= 0; x = s_parent[x]) {
#pragma unroll
          for (int w = 0; w < kMaskWords; ++w)
            if ((x >> 5) == w) a[w] |= 1u << (x & 31);
          ++depth;
        }
        --depth;
        if (depth > p.max_depth) report(p.status, DFV_DEV_DEPTH);
        atomicMax(&s_maxdepth, depth);
      }
#pragma unroll
      for (int w = 0; w < kMaskWords; ++w) s_anc[w][tid] = a[w];
      s_lo[tid] = p.window > 0 ? C + depth - p.window + 1 : INT32_MIN;
      s_m[tid] = kNoRef;
    }
    named_sync(4, 256);
    const int lo_all = p.window > 0 ? C + s_maxdepth - p.window + 1 : INT32_MIN;
    const float sc = p.scale * kLog2eF * qs;
    float l[HC];
#pragma unroll
    for (int c = 0; c < HC; ++c) l[c] = 0.0f;
    const uint32_t t_s = tmem + lanes + A::kTS + cg * HC;
    const uint32_t t_o = tmem + lanes + A::kTO + cg * HC;
    const float4* m4 = reinterpret_cast<const float4*>(s_m + cg * HC);

    for (int i = 0; i < n; ++i) {
      // this lane's key
      const bool bf = has_tree && i == n - 1;
      const int b = fb + 2 * (c0 + i);
      float a = 0.0f, lv = 0.0f, iv = 0.0f;
      int pos;
      bool live;
      if (!bf) {
        const int kb = b + (key >> 6);
        live = kb < open;
        pos = kb * kBlk + (key & 63);
        if (live) {
          const int64_t at = static_cast<int64_t>(h) * p.nblk + kb;
          a = __ldg(p.c.k_scale + at) * sc;
          const float sv = fmaxf(__ldg(p.c.v_scale + at), 7.1054274e-15f);   // 2^-47
          lv = log2f(sv);
          iv = __fdividef(1.0f, sv);
        }
      } else {
        live = key < T + p.n_nodes;
        pos = key < T ? open * kBlk + key : INT32_MAX;
      }
      ok = ok && role_wait(&b_sfull, i & 1, &s_dead);
      ok = __all_sync(0xFFFFFFFFu, ok);   // the TMEM loads are warp-wide
      tc::fence_after_sync();
      bool bad = false;
      if (bf) {   // the key's scales were written with the operands
        ok = ok && role_wait(&b_khat, i & 1, &s_dead) && role_wait(&b_vhat, i & 1, &s_dead);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (ok && live) {
          a = s_ksc[key] * sc;
          lv = static_cast<float>(s_vexp[key]);
          iv = pow2i(-s_vexp[key]);
          bad = s_badk[key] || s_badv[key];
        }
      }
      float x[HC];
      if (ok) tc::TmemIo<HC>::load(t_s, reinterpret_cast<uint32_t*>(x));
      const bool masked = bf || b + 2 > open || b * kBlk < lo_all;
      // keys this lane's column may not see
      auto mask = [&]() {
        if (!masked) return;
        const int t = key - T;   // tree node of the slot
#pragma unroll
        for (int c = 0; c < HC; ++c) {
          bool see = live && pos >= s_lo[cg * HC + c];
          if (bf && t >= 0) see = live && ((s_anc[t >> 5][cg * HC + c] >> (t & 31)) & 1u);
          if (!see) x[c] = -INFINITY;
        }
      };
      auto exponents = [&]() {
        float top = -INFINITY;
#pragma unroll
        for (int c = 0; c < HC; c += 4) {
          const float4 m = m4[c / 4];
          x[c] = fmaf(x[c], a, lv - m.x);
          x[c + 1] = fmaf(x[c + 1], a, lv - m.y);
          x[c + 2] = fmaf(x[c + 2], a, lv - m.z);
          x[c + 3] = fmaf(x[c + 3], a, lv - m.w);
        }
        mask();
#pragma unroll
        for (int c = 0; c < HC; ++c) top = fmaxf(top, x[c]);
        return top;
      };
      if (!named_sync_and(5 + cg, 128, !(exponents() > kRaise) && ok)) {
        // some column outgrew its reference (or a wait gave up)
        if (!named_sync_and(5 + cg, 128, ok)) break;
        tc::TmemIo<HC>::load(t_s, reinterpret_cast<uint32_t*>(x));
#pragma unroll
        for (int c = 0; c < HC; ++c) x[c] = fmaf(x[c], a, lv);
        mask();
#pragma unroll
        for (int c = 0; c < HC; ++c) {
          float m;
          asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(x[c]));
          if (lane == 0) s_red[warp & 3][cg * HC + c] = m;
        }
        named_sync(5 + cg, 128);
        if ((warp & 3) == 0) {
          for (int c = cg * HC + lane; c < (cg + 1) * HC; c += 32) {
            const float was = s_m[c];
            const float m = fmaxf(fmaxf(fmaxf(s_red[0][c], s_red[1][c]),
                                        fmaxf(s_red[2][c], s_red[3][c])), was);
            s_m[c] = m;
            s_f[c] = tc::ex2(was - m);
          }
        }
        if (i > 0) ok = role_wait(&b_pv[(i - 1) & 1], ((i - 1) >> 1) & 1, &s_dead);
        ok = named_sync_and(5 + cg, 128, ok);
        if (!ok) break;
        tc::fence_after_sync();
#pragma unroll
        for (int c = 0; c < HC; ++c) l[c] *= s_f[cg * HC + c];
        if (i > 0) {
#pragma unroll
          for (int hh = 0; hh < A::kHalves; ++hh) {
            tc::TmemIo<HC>::load(t_o + hh * R, reinterpret_cast<uint32_t*>(x));
#pragma unroll
            for (int c = 0; c < HC; ++c) x[c] *= s_f[cg * HC + c];
            tc::TmemIo<HC>::store(t_o + hh * R, reinterpret_cast<const uint32_t*>(x));
            tc::store_wait();
          }
        }
        tc::TmemIo<HC>::load(t_s, reinterpret_cast<uint32_t*>(x));
        exponents();
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
      if (A::kPBufs == 2 && i >= 2) ok = role_wait(&b_pv[pb], ((i - 2) >> 1) & 1, &s_dead);
      if (A::kPBufs == 1 && i >= 1) ok = role_wait(&b_pv[pb ^ 1], ((i - 1) >> 1) & 1, &s_dead);
      if (ok) {
        uint8_t* dst = sP + (A::kPBufs == 2 ? pb : 0) * A::kPBytes;
#pragma unroll
        for (int j = 0; j < HC / 8; ++j) {
          uint32_t o[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float p0 = tc::ex2(x[8 * j + 2 * e]), p1 = tc::ex2(x[8 * j + 2 * e + 1]);
            l[8 * j + 2 * e] = fmaf(p0, iv, l[8 * j + 2 * e]);
            l[8 * j + 2 * e + 1] = fmaf(p1, iv, l[8 * j + 2 * e + 1]);
            o[e] = pack_half2(p0, p1);
          }
          *reinterpret_cast<uint4*>(dst + tc::sw128_offset(key, cg * (HC / 8) + j, kAtKeys)) =
              make_uint4(o[0], o[1], o[2], o[3]);
        }
      }
      fence_proxy_async_smem();
      if (__all_sync(0xFFFFFFFFu, ok) && lane == 0) mbar_arrive(&b_p[pb]);
    }
    // ---- the unit's result
    if (ok && n > 0) ok = role_wait(&b_pv[(n - 1) & 1], ((n - 1) >> 1) & 1, &s_dead);
    ok = named_sync_and(5 + cg, 128, ok);
    tc::fence_after_sync();
#pragma unroll
    for (int c = 0; c < HC; ++c) {
      float s = l[c];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
      if (lane == 0) s_red[warp & 3][cg * HC + c] = s;
    }
    named_sync(5 + cg, 128);
    const int64_t all_rows = static_cast<int64_t>(p.n_nodes) * p.hq;
    if ((warp & 3) == 0) {
      for (int c = cg * HC + lane; c < (cg + 1) * HC; c += 32) {
        const float s = (s_red[0][c] + s_red[1][c]) + (s_red[2][c] + s_red[3][c]);
        const float lse = s == 0.0f || !ok ? -INFINITY : s_m[c] + log2f(s);
        s_f[c] = s == 0.0f ? 0.0f : 1.0f / s;
        if (c < n_rows) {
          if (p.splits > 1) p.part_lse[split * all_rows + s_row[c]] = lse;
          else if (p.lse) p.lse[s_row[c]] = lse * kLn2F;
        }
      }
    }
    named_sync(5 + cg, 128);
    if (ok && n > 0) {
#pragma unroll
      for (int hh = 0; hh < A::kHalves; ++hh) {
        float x[HC];
        tc::TmemIo<HC>::load(t_o + hh * R, reinterpret_cast<uint32_t*>(x));
        const int d = hh * 128 + key;
        if (d < D) {
#pragma unroll
          for (int c = 0; c < HC; ++c) {
            const int col = cg * HC + c;
            if (col >= n_rows) continue;
            const float o = x[c] * s_f[col];
            const int64_t at = static_cast<int64_t>(s_row[col]) * D + d;
            if (p.splits > 1) p.part_o[split * all_rows * D + at] = o;
            else if (p.out_bf16) static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(o);
            else static_cast<float*>(p.out)[at] = o;
          }
        }
      }
    }
    tc::fence_before_sync();
  }
  __syncwarp();
  __syncthreads();
  if (warp == 16) {
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

template <int D>
__global__ void __launch_bounds__(kMergeThreads)
    kv8_merge_kernel(int splits, const float* part_o, const float* part_lse, void* out,
                     int out_bf16, float* lse) {
  constexpr int kV = D / 4, kG = kMergeThreads / kV;   // float4 of a row; groups of splits
  __shared__ float s_w[kMaxSplits];
  __shared__ float4 s_o[kG][kV];
  const int tid = threadIdx.x, lane = tid & 31;
  const int64_t row = blockIdx.x, rows = gridDim.x;
  grid_dep_wait();
  float m = -INFINITY;
  for (int s = lane; s < splits; s += 32) m = fmaxf(m, part_lse[s * rows + row]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  float total = 0.0f;
  for (int s = lane; s < splits; s += 32) {
    const float v = part_lse[s * rows + row];
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
    const float4 v = reinterpret_cast<const float4*>(part_o + (s * rows + row) * D)[tid % kV];
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
    if (out_bf16) {
      const __nv_bfloat162 lo = __floats2bfloat162_rn(a.x, a.y), hi = __floats2bfloat162_rn(a.z, a.w);
      reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(out) + row * D)[tid] =
          make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
    } else {
      reinterpret_cast<float4*>(static_cast<float*>(out) + row * D)[tid] = a;
    }
  }
  if (tid == 0 && lse)
    lse[row] = total == 0.0f ? -INFINITY : (m + log2f(total)) * kLn2F;
}

// ---------------------------------------------------------------- host

struct AttnPlan {
  int tiles, rows_tile, r, splits;
};

constexpr int kMaxRows = 80;   // query rows of a tile (TMEM columns at D = 256)

// Tiles of at most 80 rows, as even as they come. Slices: a unit costs its
// chunks plus about two for its start and end, and the SMs take units in
// waves; the count with the least time, the fewest of equals.
static AttnPlan attn_plan(int n_nodes, int hq, int hkv, int window, int capacity) {
  AttnPlan pl;
  const int rows = n_nodes * (hq / hkv);
  pl.tiles = (rows + kMaxRows - 1) / kMaxRows;
  pl.rows_tile = (rows + pl.tiles - 1) / pl.tiles;
  pl.r = (pl.rows_tile + 15) / 16 * 16;
  const int span = window > 0 && window < capacity ? window : capacity;
  const int chunks = span / kAtKeys + 2;
  const int64_t units = static_cast<int64_t>(hkv) * pl.tiles;
  const int sms = sm_count();
  const int most = chunks < kMaxSplits ? chunks : kMaxSplits;
  int64_t best = INT64_MAX;
  pl.splits = 1;
  for (int s = 1; s <= most && (s == 1 || units * s <= 4 * sms); ++s) {
    const int64_t waves = (units * s + sms - 1) / sms;
    const int64_t cost = waves * ((chunks + s - 1) / s + 2);
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

static size_t attn_ws_bytes(const AttnPlan& pl, int n_nodes, int hq, int d) {
  if (pl.splits == 1) return 256;
  return static_cast<size_t>(pl.splits) * n_nodes * hq * (d + 4) * sizeof(float) + 256;
}

template <int D, int R>
static dfv_status attn_launch(const AttnParams& p, int units, cudaStream_t stream) {
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
  kv8_attn_kernel<D, R><<<units * p.splits, kAtThreads, A::kBytes, stream>>>(p);
  if (cudaGetLastError() != cudaSuccess) return DFV_ERR_CUDA;
  if (p.splits == 1) return DFV_OK;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.n_nodes * p.hq);
  cfg.blockDim = dim3(kMergeThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv8_merge_kernel<D>, p.splits,
                            static_cast<const float*>(p.part_o),
                            static_cast<const float*>(p.part_lse), p.out, p.out_bf16,
                            p.lse) == cudaSuccess
             ? DFV_OK
             : DFV_ERR_CUDA;
}

template <int D>
static dfv_status attn_launch_r(const AttnParams& p, int r, int units, cudaStream_t stream) {
  switch (r) {
    case 16: return attn_launch<D, 16>(p, units, stream);
    case 32: return attn_launch<D, 32>(p, units, stream);
    case 48: return attn_launch<D, 48>(p, units, stream);
    case 64: return attn_launch<D, 64>(p, units, stream);
    default: return attn_launch<D, 80>(p, units, stream);
  }
}

}  // namespace dfv

extern "C" size_t dfv_kv8_attn_workspace_bytes(int n_nodes, int n_q_heads, int n_kv_heads,
                                               int head_dim, int window, int cache_capacity) {
  using namespace dfv;
  if (!attn_shape_ok(n_nodes, n_q_heads, n_kv_heads, head_dim, window, cache_capacity)) return 0;
  return attn_ws_bytes(attn_plan(n_nodes, n_q_heads, n_kv_heads, window, cache_capacity), n_nodes,
                       n_q_heads, head_dim);
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
  const AttnPlan pl = attn_plan(n_nodes, n_q_heads, hkv, window, cache->capacity);
  if (pl.splits > 1) {
    if (!workspace || !aligned(workspace, 256)) return DFV_ERR_INVALID;
    if (workspace_bytes < attn_ws_bytes(pl, n_nodes, n_q_heads, d)) return DFV_ERR_WORKSPACE;
  }
  AttnParams p = {};
  p.c = *cache;
  p.nblk = kv8_blocks(cache->capacity);
  p.n_nodes = n_nodes;
  p.max_depth = max_depth;
  p.hq = n_q_heads;
  p.group = n_q_heads / hkv;
  p.window = window;
  p.rows = n_nodes * p.group;
  p.tiles = pl.tiles;
  p.rows_tile = pl.rows_tile;
  p.splits = pl.splits;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.tree_k = static_cast<const __nv_bfloat16*>(tree_k);
  p.tree_v = static_cast<const __nv_bfloat16*>(tree_v);
  p.parent = parent;
  p.scale = scale > 0.0f ? scale : 1.0f / sqrtf(static_cast<float>(d));
  p.out = out;
  p.out_bf16 = out_dtype == DFV_DTYPE_BF16;
  p.lse = lse;
  p.part_o = static_cast<float*>(workspace);
  p.part_lse = p.part_o + static_cast<size_t>(pl.splits) * n_nodes * n_q_heads * d;
  p.status = status;
  const int units = hkv * pl.tiles;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  switch (d) {
    case 64: return attn_launch_r<64>(p, pl.r, units, s);
    case 128: return attn_launch_r<128>(p, pl.r, units, s);
    default: return attn_launch_r<256>(p, pl.r, units, s);
  }
}
