// The attention weight that each cached key receives from the last committed
// rows, summed over the rows and the query heads of the key's group:
//
//   weights[h][j] = decay * prev[h][j] + sum_{s, g} exp(scale q_{s,hg} . k_j - lse_{s,hg})
//
// over the rows s that see key j. Keys are the M dimension of the product (S^T
// = K^ Q^T, 128 keys x up to 128 query rows), so a key is a lane of TMEM: the
// sum over query rows is a sum over a thread's own columns, without any exchange
// between lanes.
//
// The weights are f32 results, so K^ has to be exact: a Q4_0 value (code - 8) d
// has 14 bits and binary16 holds 11. It is split into hi = rn16((code - 8) d)
// and lo = (code - 8) d - hi, which fits binary16 exactly, and both are
// multiplied (weights off by 1.4e-4 with hi alone, by 1e-6 so). F16 rows are
// exact. Query rows are scaled by a power of two each, which the exponent's
// factor takes back.
//
// Up to 16 query rows of a KV head (decoding) leave TMEM room for the sums of
// each block of 32 dims apart: then K^ is the codes' integers alone, half the
// products and stores and a third of the conversion, and a key's block scales
// are factors of its lane's sums (131060 keys, 4 heads of 256, 6 rows each:
// 22.8 us, by hi and lo 34).
//
// A CTA works through a run of 128-key chunks of (at most a few) heads, in parts
// of up to 256 dims. Q4_0: one warp copies raw rows into a ring, two groups of four
// convert parts in turn into TMEM, the product's A operand. F16: the two groups
// copy parts straight into swizzled tiles, A from shared memory. One warp
// issues the products; two groups of four warps take turns at the chunks' sums.
//
// Bound by issue: hand-offs and conversion for few rows (one row over 131060
// Q4_0 keys, 4 heads of 256: 22.5 us, 3.4 TB/s; nine rows over 61440
// 17.4), the sums for many (65 nodes, 32 / 8 heads of 128, 32791 F16
// keys: 35 us, 25 % of the products' rate; 6 of them build the query rows).

#include <atomic>

#include "common.cuh"
#include "tc.cuh"
#include "tmem_io.cuh"

namespace dfv {

constexpr int kWtKeys = 128;
constexpr int kWtMma = 16, kWtRaw = 17;      // warps 0-7: sums, 8-15: operands
constexpr int kWtThreads = 18 * 32;

// F16 (rows by slices or not); Q4_0: hi and lo, or block by block
enum WeightMode { kModeF16, kModeSliced, kModeSplit, kModeBlocks };

template <int D, int kMode>
struct WeightShape {
  static constexpr bool kQ4 = kMode == kModeSplit || kMode == kModeBlocks;
  static constexpr bool kBlocks = kMode == kModeBlocks, kSliced = kMode == kModeSliced;
  // Query rows of a tile, at most. Sliced: in two slices of scores, three of
  // which are in TMEM, so that K is read once for as many rows as fit shared memory
  // (260 rows of a head, 61440 F16 keys: 54 us, in three slices 57; before the
  // sums were faster, 73 for 78 in two tiles).
  static constexpr int kRows = kBlocks ? 16 : kQ4 || D == 256 ? 128 : kSliced ? 288 : 256;
  static constexpr int kRowBytes = kQ4 ? D / 32 * 18 : D * 2;
  // Parts of a chunk: with Q4_0 as many times 64 dims as leave TMEM room for two
  // parts, F16 128 dims (handing a part over costs as much as converting 64 dims:
  // one row over 131060 keys 22.8 us, by 128 dims 25.9, by 64 30.7).
  static constexpr int kHalves = kBlocks ? D / 64 : D >= 128 ? 2 : 1;
  static constexpr int kParts = D / 64 / kHalves;
  static constexpr int kHalfCols = kBlocks ? 32 : 64;         // Q4_0: TMEM columns
  static constexpr int kPartCols = kHalves * kHalfCols;
  static constexpr int kPartBytes = kHalves * kWtKeys * 128;  // F16: tiles of 64 dims
  static constexpr int kRing = kBlocks ? 2 * kParts : kQ4 ? 256 / kPartCols : 8 / kHalves;
  static constexpr int kStages = 4;                           // Q4_0: raw chunks
  static constexpr int kStage = (kWtKeys * kRowBytes + 16 + 127) / 128 * 128;
  static constexpr int kQBytes = kRows * D * 2;
  static constexpr int kBytes = kQBytes + (kQ4 ? kStages * kStage : kRing * kPartBytes) + 1024;
  // Scores: two buffers; sliced as many slices as fit, at most eight
  static constexpr uint32_t kTS = kQ4 ? 256 : 0;
  static constexpr int kSCols = kBlocks ? D / 32 * kRows : kSliced ? 128 : kRows;
  static_assert(kTS + 2 * kSCols <= 512, "TMEM columns");
  static_assert(kBytes <= 220 * 1024, "shared memory");
};

template <int kN> struct Columns {
  static constexpr int value = kN;
};

struct WeightParams {
  int n_rows, hq, hkv, group, window, capacity;
  uint32_t group_m;   // ceil(2^32 / group) where r / group = umulhi(r, group_m) for all rows, or 0
  const int32_t* ctx_len;
  const uint8_t* k;
  const __nv_bfloat16* q;
  const float* lse;
  const int32_t *path, *accept_len;
  float scale, decay;
  const float* prev;
  float* weights;
  uint32_t* status;
};

// Place of dim c of a block of 32 in the operands' K order (Q4_0): a word of four code
// bytes gives pairs (bytes 0, 2 low), (0, 2 high), (1, 3 low), (1, 3 high).
// Eight consecutive places are word w's dims 4w + {0, 2, 16, 18, 1, 3, 17, 19}.

template <int D, int kMode>
__global__ void __launch_bounds__(kWtThreads, 1)
    kv_weights_kernel(const __grid_constant__ WeightParams p) {
  using W = WeightShape<D, kMode>;
  constexpr bool kQ4 = W::kQ4, kBlocks = W::kBlocks, kSliced = W::kSliced;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* sQ = smem;
  uint8_t* sK = smem + W::kQBytes;                    // raw rows, or tiles
  __shared__ uint64_t b_raw[4], b_read[4];            // raw rows landed, read
  __shared__ uint64_t b_part[8], b_free[8];           // operand part written, multiplied
  __shared__ uint64_t b_s[8], b_sfree[8];             // scores there, read
  __shared__ uint64_t b_q, b_qfree, b_end;            // query rows there, multiplied
  __shared__ uint32_t s_tmem;
  __shared__ volatile int s_dead;
  // of a tile's columns, two tiles in turn: the exponent's slope and offset,
  // and the first and last position that is seen
  __shared__ __align__(16) float s_slope[2][W::kRows], s_off[2][W::kRows];
  __shared__ __align__(16) int s_first[2][W::kRows], s_last[2][W::kRows];
  // Block scales of four chunks' keys in turn. They are written once the part's
  // place is free: the chunk two before has been multiplied then, which waited
  // for the sums of the chunk four before.
  __shared__ __half s_scale[kBlocks ? 4 : 1][kBlocks ? D / 32 : 1][kBlocks ? kWtKeys : 1];

  const int tid = threadIdx.x, lane = tid & 31;
  const int warp =
      static_cast<int>(__reduce_max_sync(0xFFFFFFFFu, static_cast<unsigned>(tid >> 5)));
  if (tid == 0) {
    for (int i = 0; i < 4; ++i) {
      mbar_init(&b_raw[i], 1);
      mbar_init(&b_read[i], W::kParts == 1 ? 4 : 8);   // the groups that read it
    }
    for (int i = 0; i < 8; ++i) {
      mbar_init(&b_part[i], 4);
      mbar_init(&b_free[i], 1);
    }
    for (int i = 0; i < 8; ++i) {
      mbar_init(&b_s[i], kBlocks ? 2 : 1);
      mbar_init(&b_sfree[i], 4);
    }
    mbar_init(&b_q, 8);
    mbar_init(&b_qfree, 1);
    mbar_init(&b_end, 1);
    s_dead = 0;
    fence_mbar_init();
  }
  grid_dep_wait();
  grid_dep_launch_dependents();   // (after the wait: see common.cuh)
  if (warp == kWtMma) tc::tmem_alloc(&s_tmem, 512);

  // ---- the problem, the same in every thread
  int C = __reduce_max_sync(0xFFFFFFFFu, *p.ctx_len);
  if (C < 0 || C > p.capacity) {
    if (tid == 0) report(p.status, DFV_DEV_CTX);
    C = max(0, min(C, p.capacity));
  }
  int n = p.n_rows;
  if (p.accept_len) {
    const int L = __reduce_max_sync(0xFFFFFFFFu, *p.accept_len);
    if ((L < 0 || L > n) && tid == 0) report(p.status, DFV_DEV_BAD_PATH);
    n = max(0, min(L, n));
  }
  const int rows = n * p.group;                       // query rows of a KV head
  const int tiles = (rows + W::kRows - 1) / W::kRows;
  // slices of a tile, and their columns, balanced, in steps of 16
  const int tile_rows = tiles == 0 ? 1 : (rows + tiles - 1) / tiles;
  const int slices = kSliced ? (tile_rows + 255) / 256 : 1;
  const int RS = ((tile_rows + slices - 1) / slices + 15) / 16 * 16, R = slices * RS;
  // places of slices of scores, taken in turn: slice number i has place i % places
  const uint32_t places = kSliced ? min(8, 512 / RS) : 2;
  const uint32_t place_cols = kSliced ? RS : W::kSCols;
  // place and turn (how often it was taken) of a chunk's first slice, from
  // those of a chunk before, and of the next slice
  auto skip = [&](uint32_t& place, uint32_t& turn, int by) {
    place += by;
    while (place >= places) place -= places, ++turn;
  };
  // positions: row s stands at C - n + s; chunks [fc, lc) are seen by some row
  const int at0 = C - n;
  const int lc = tiles == 0 ? 0 : (C + kWtKeys - 1) / kWtKeys;
  const int fc = p.window > 0 ? min(lc, max(0, at0 - p.window + 1) / kWtKeys) : 0;
  const int64_t all = static_cast<int64_t>(p.hkv) * (lc - fc);
  const int64_t u0 = all * blockIdx.x / gridDim.x, u1 = all * (blockIdx.x + 1) / gridDim.x;
  const int per_head = max(1, lc - fc);

  // Runs of chunks of one head, each for every tile: f(head, first chunk, last
  // chunk + 1, tile) in the same order in every role; false ends.
  auto runs = [&](auto f) {
    for (int64_t u = u0; u < u1;) {
      const int h = static_cast<int>(u / per_head), c = static_cast<int>(u % per_head);
      const int m = static_cast<int>(min(u1 - u, static_cast<int64_t>(per_head - c)));
      for (int t = 0; t < tiles; ++t)
        if (!f(h, fc + c, fc + c + m, t)) return;
      u += m;
    }
  };
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = s_tmem;
  const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;   // quadrant's first lane << 16

  if (warp == kWtRaw) {
    // ------------------------------------------------------ raw rows (Q4_0)
    bool ok = true;
    int k = 0;   // chunks so far
    fence_proxy_async_global();   // what earlier kernels wrote, to the copy engine
    runs([&](int h, int c0, int c1, int) {
      for (int c = c0; kQ4 && c < c1; ++c, ++k) {
        const int st = k % W::kStages;
        if (k >= W::kStages) {
          ok = role_wait(&b_read[st], (k / W::kStages - 1) & 1, &s_dead);
          ok = __all_sync(0xFFFFFFFFu, ok);
          if (!ok) return false;
        }
        const int live = min(kWtKeys, C - c * kWtKeys);
        const int64_t from = (static_cast<int64_t>(h) * p.capacity + c * kWtKeys) * W::kRowBytes;
        uint8_t* dst = sK + st * W::kStage;
        // one piece, from the 16-byte boundary before its start; what is
        // behind the last boundary by words
        const int64_t a = from & ~static_cast<int64_t>(15);
        const int64_t e = from + static_cast<int64_t>(live) * W::kRowBytes;
        const int64_t b = e & ~static_cast<int64_t>(15);
        if (lane < static_cast<int>(e - b) / 4)
          *reinterpret_cast<uint32_t*>(dst + (b - a) + lane * 4) =
              *reinterpret_cast<const uint32_t*>(p.k + b + lane * 4);
        __syncwarp();
        if (lane == 0) {
          mbar_arrive_expect_tx(&b_raw[st], static_cast<uint32_t>(b - a));
          if (b > a) bulk_g2s(dst, p.k + a, static_cast<uint32_t>(b - a), &b_raw[st]);
        }
      }
      return true;
    });
    // copies that nobody waits for any more must still land
    if (s_dead)
      for (int i = max(0, k - W::kStages); i < k; ++i)
        mbar_wait_bounded(&b_raw[i % W::kStages], (i / W::kStages) & 1);
  } else if (warp == kWtMma) {
    // ------------------------------------------------------ products
    bool ok = true;
    int k = 0, part = 0, run = 0;
    uint32_t place0 = 0, turn0 = 0;   // of the chunk's first slice
    const uint32_t idesc = tc::idesc_f16(128, 0) | (static_cast<uint32_t>(RS >> 3) << 17);
    const uint64_t qd = tc::smem_desc_sw128(smem_u32(sQ), 1024);
    const uint64_t q_block = static_cast<uint64_t>(R * 128) >> 4;   // 64 dims of all rows
    auto all_wait = [&](uint64_t* bar, uint32_t parity) {
      const bool got = __all_sync(0xFFFFFFFFu, role_wait(bar, parity, &s_dead));
      tc::fence_after_sync();
      return got;
    };
    runs([&](int, int c0, int c1, int) {
      ok = all_wait(&b_q, run & 1);
      for (int c = c0; ok && c < c1; ++c, ++k) {
        if constexpr (!kSliced) place0 = k & 1, turn0 = k >> 1;
        for (int i = 0; ok && i < W::kParts; ++i, ++part) {
          const int slot = part % W::kRing;
          uint32_t place = place0, turn = turn0;
          // (a chunk's slices are at most as many as the places)
          for (int sl = 0; ok && sl < slices; ++sl) {
            if (i == 0 && turn > 0) ok = all_wait(&b_sfree[place], (turn - 1) & 1);
            if (ok && sl == 0) ok = all_wait(&b_part[slot], (part / W::kRing) & 1);
            if (!ok) break;
            if (tc::elect_one()) {
              const uint32_t d = tmem + W::kTS + place * place_cols;
              if constexpr (kQ4) {
#pragma unroll
                for (int hh = 0; hh < W::kHalves; ++hh) {
                  const int g = i * W::kHalves + hh;   // which 64 dims
                  const uint32_t a = tmem + slot * W::kPartCols + hh * W::kHalfCols;
                  if constexpr (kBlocks) {
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)   // two steps a block
                      tc::mma_f16_ts(d + (2 * g + (kk >> 1)) * W::kRows, a + kk * 8,
                                     qd + g * q_block + kk * 2, idesc, kk & 1);
                  } else {
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)   // hi, then lo
                      tc::mma_f16_ts(d, a + kk * 8, qd + g * q_block + (kk & 3) * 2, idesc,
                                     g > 0 || kk > 0 ? 1u : 0u);
                  }
                }
              } else {
                const uint64_t a0 =
                    tc::smem_desc_sw128(smem_u32(sK + slot * W::kPartBytes), 1024);
#pragma unroll
                for (int hh = 0; hh < W::kHalves; ++hh) {
                  const int g = i * W::kHalves + hh;   // which 64 dims
                  const uint64_t a = a0 + hh * (kWtKeys * 128 >> 4);
                  const uint64_t q = qd + g * q_block + sl * RS * 8;
#pragma unroll
                  for (int kk = 0; kk < 4; ++kk)
                    tc::mma_f16(d, a + kk * 2, q + kk * 2, idesc, g > 0 || kk > 0 ? 1u : 0u);
                }
              }
              if (sl == slices - 1) tc::commit(&b_free[slot]);
              if (i == W::kParts - 1) tc::commit(&b_s[place]);
              // (an arrival of its own: a commit orders the products, not the scales)
              if (kBlocks && i == W::kParts - 1) mbar_arrive(&b_s[place]);
            }
            __syncwarp();
            if constexpr (kSliced) skip(place, turn, 1);
          }
        }
        if constexpr (kSliced) skip(place0, turn0, slices);
      }
      if (!ok) return false;
      if (tc::elect_one()) tc::commit(&b_qfree);
      __syncwarp();
      ++run;
      return true;
    });
    // products in flight must end before TMEM is freed
    if (!ok) s_dead = 1;
    if (tc::elect_one()) tc::commit(&b_end);
    __syncwarp();
    mbar_wait_bounded(&b_end, 0);
  } else if (warp >= 8) {
    // ------------------------------------------------------ operands
    // Two groups of four warps, each with every other part.
    const int set = (warp >> 2) & 1, slot = (warp & 3) * 32 + lane;   // key of the chunk
    bool ok = true;
    int k = 0, part = 0;
    auto take = [&]() {   // the part's place is free
      if (part >= W::kRing)
        ok = role_wait(&b_free[part % W::kRing], (part / W::kRing - 1) & 1, &s_dead);
      ok = __all_sync(0xFFFFFFFFu, ok);   // the TMEM stores are warp-wide
    };
    if constexpr (kQ4) {
      runs([&](int h, int c0, int c1, int) {
        for (int c = c0; ok && c < c1; ++c, ++k) {
          if (W::kParts == 1 && (part & 1) != set) {
            ++part;
            continue;
          }
          const int st = k % W::kStages;
          ok = __all_sync(0xFFFFFFFFu, role_wait(&b_raw[st], (k / W::kStages) & 1, &s_dead));
          if (!ok) break;
          // rows of 36 or 72 bytes: the piece began at a 16-byte boundary
          const uint8_t* row = sK + st * W::kStage + slot * W::kRowBytes;
          if (D < 256)
            row += ((static_cast<int64_t>(h) * p.capacity + c * kWtKeys) * W::kRowBytes) & 15;
          // 64 dims are two blocks of 18 bytes, nine words, read by pieces of D / 16
          // bytes (without bank conflicts: the rows are nine of them apart).
          constexpr int kE = D / 64;                  // words of a piece
          constexpr int kLast = (W::kParts - 1) & ~1; // first of the last two parts
#pragma unroll
          for (int i = 0; i < W::kParts; ++i, ++part) {
            if ((part & 1) != set) continue;
            const uint32_t t = tmem + lanes + (part % W::kRing) * W::kPartCols;
#pragma unroll
            for (int hh = 0; hh < W::kHalves; ++hh) {
              constexpr int kPieces = D == 256 ? 3 : D == 128 ? 5 : 9;
              const int g = i * W::kHalves + hh;      // which 64 dims
              const int p0 = 9 * g / kE;              // the piece with the first word
              uint32_t in[kPieces * kE + 1];
#pragma unroll
              for (int e = 0; e < kPieces; ++e) {
                if constexpr (D == 256) {
                  const uint4 v = *reinterpret_cast<const uint4*>(row + (p0 + e) * 16);
                  in[4 * e] = v.x, in[4 * e + 1] = v.y, in[4 * e + 2] = v.z, in[4 * e + 3] = v.w;
                } else if constexpr (D == 128) {
                  const uint2 v = *reinterpret_cast<const uint2*>(row + (p0 + e) * 8);
                  in[2 * e] = v.x, in[2 * e + 1] = v.y;
                } else {
                  in[e] = *reinterpret_cast<const uint32_t*>(row + (p0 + e) * 4);
                }
              }
              if (i >= kLast && hh == W::kHalves - 1) {
                // the group's last codes are in registers
                __syncwarp();
                if (lane == 0) mbar_arrive(&b_read[st]);
              }
              const uint32_t* words = in + (9 * g - p0 * kE);
              uint32_t hi[32], lo[kBlocks ? 1 : 32];
#pragma unroll
              for (int b = 0; b < 2; ++b) {
                // codes follow the scale: words of the first block are 2 bytes off
                const uint32_t* w = words + 4 * b;
                const uint32_t sc = b == 0 ? w[0] & 0xFFFFu : w[0] >> 16;
                const uint32_t d2 = sc | (sc << 16);
                const __half2 d = *reinterpret_cast<const __half2*>(&d2);
                const __half2 low = __float2half2_rn(1032.0f);    // 1024 + 8
                const __half2 high = __float2half2_rn(1152.0f);   // 1024 + 16 * 8
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  const uint32_t x = b == 0 ? __funnelshift_r(w[j], w[j + 1], 16) : w[j + 1];
#pragma unroll
                  for (int e = 0; e < 4; ++e) {
                    // 0x6400 | code is 1024 + code; block by block a high nibble
                    // stays where it is: 0x6400 | code << 4 is 1024 + 16 code
                    const bool up = kBlocks && (e & 1);
                    const uint32_t y = up ? ((x >> (4 * e - 4)) & 0x00F000F0u) | 0x64006400u
                                          : ((x >> (4 * e)) & 0x000F000Fu) | 0x64006400u;
                    const __half2 v =
                        __hsub2(*reinterpret_cast<const __half2*>(&y), up ? high : low);
                    if constexpr (kBlocks) {
                      hi[b * 16 + j * 4 + e] = *reinterpret_cast<const uint32_t*>(&v);
                    } else {
                      const __half2 a = __hmul2(v, d);
                      const __half2 r = __hfma2(v, d, __hneg2(a));
                      hi[b * 16 + j * 4 + e] = *reinterpret_cast<const uint32_t*>(&a);
                      lo[b * 16 + j * 4 + e] = *reinterpret_cast<const uint32_t*>(&r);
                    }
                  }
                }
              }
              if (hh == 0) take();
              if (!ok) break;
              if (hh == 0) tc::fence_after_sync();
              if constexpr (kBlocks) {   // (not before the place is free)
                s_scale[k & 3][2 * g][slot] = __ushort_as_half(words[0] & 0xFFFFu);
                s_scale[k & 3][2 * g + 1][slot] = __ushort_as_half(words[4] >> 16);
              }
              tc::TmemIo<32>::store(t + hh * W::kHalfCols, hi);
              if constexpr (!kBlocks) tc::TmemIo<32>::store(t + hh * W::kHalfCols + 32, lo);
            }
            if (!ok) break;
            tc::store_wait();
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&b_part[part % W::kRing]);
          }
        }
        return ok;
      });
    } else {
      // A part: 128 rows of 128 bytes, eight 16-byte pieces a thread; a group
      // has up to kLag + 1 parts in flight.
      constexpr int kLag = W::kRing / 2 - 1;
      int issued = 0, given = 0;   // of the group's parts
      auto give = [&]() {          // this thread's oldest copies have landed
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&b_part[(2 * given + set) % W::kRing]);
        ++given;
      };
      const int t = (warp & 3) * 32 + lane;
      runs([&](int h, int c0, int c1, int) {
        for (int c = c0; ok && c < c1; ++c) {
          const int live = min(kWtKeys, C - c * kWtKeys);
          const uint8_t* src =
              p.k + (static_cast<int64_t>(h) * p.capacity + c * kWtKeys) * W::kRowBytes;
          for (int i = 0; i < W::kParts; ++i, ++part) {
            if ((part & 1) != set) continue;
            take();
            if (!ok) break;
            uint8_t* dst = sK + (part % W::kRing) * W::kPartBytes;
#pragma unroll
            for (int e = 0; e < 8 * W::kHalves; ++e) {
              const int r = (t >> 3) + e % 8 * 16, j = (t & 7) + e / 8 * 8;
              if (r < live)
                cp_async16(dst + tc::sw128_offset(r, j, kWtKeys),
                           src + static_cast<int64_t>(r) * W::kRowBytes +
                               i * (W::kHalves * 128) + j * 16);
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
            ++issued;
            if (issued > kLag) {
              asm volatile("cp.async.wait_group %0;" ::"n"(kLag) : "memory");
              give();
            }
          }
        }
        return ok;
      });
      asm volatile("cp.async.wait_group 0;" ::: "memory");
      while (ok && given < issued) give();
    }
  } else {
    // ------------------------------------------------------ query rows, sums
    const int grp = warp >> 2;
    bool ok = true;
    int k = 0, run = 0;
    uint32_t place = 0, turn = 0;
    skip(place, turn, grp * slices);
    runs([&](int h, int c0, int c1, int t) {
      const int r0 = t * R, live = min(R, rows - r0), tb = run & 1;
      // Query rows: D / 8 lanes each, kBatch of a lane's rows loaded together.
      // The largest magnitude of a row becomes a power of two.
      constexpr int kLanes = D / 8, kPerStep = 8 * 32 / kLanes, kBatch = 4;
      const int piece = lane % kLanes;
      uint32_t problems = 0;
      // The tile's power of two, 2^4 above its first row's: rows within 2^-8 to 1
      // of it have that one (their elements are exact down to 2^-23 of the row's
      // largest), and where all have, the exponent's slope stays in a register
      // (65 rows, 32 / 8 heads of 128 over 61440 F16 keys: 77 us, slopes read for
      // every column 82).
      int e_tile = 40;
      bool own = false;   // some row has another one
      if (!kBlocks) {
        const int step = r0 / p.group, g = r0 - step * p.group;
        const int node = p.path ? p.path[step] : step;
        if (node >= 0 && node < p.n_rows) {
          const uint4 v = *reinterpret_cast<const uint4*>(
              p.q + (static_cast<int64_t>(node) * p.hq + h * p.group + g) * D + piece * 8);
          uint32_t m = __vmaxu2(__vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu),
                                __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu));
          m = max(m & 0xFFFFu, m >> 16);
          e_tile = max(min(static_cast<int>(__reduce_max_sync(0xFFFFFFFFu, m) >> 7) + 4, 254), 40);
        }
      }
      for (int rb = 0; rb < R; rb += kBatch * kPerStep) {
        uint2 a[kBatch], b[kBatch];
        float l[kBatch];
        int s[kBatch];
        bool bad[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          // (no branches: a batch's loads are in flight together)
          const int r = rb + i * kPerStep + warp * (32 / kLanes) + lane / kLanes;
          const uint32_t at = r0 + min(r, live - 1);
          const int step = p.group_m ? static_cast<int>(__umulhi(at, p.group_m))
                                     : static_cast<int>(at) / p.group;
          const int g = static_cast<int>(at) - step * p.group;
          const int node = p.path ? p.path[step] : step;
          const bool there = node >= 0 && node < p.n_rows;
          bad[i] = r < live && !there;
          s[i] = r < live && there ? step : -1;
          const int64_t row = static_cast<int64_t>(there ? node : 0) * p.hq + h * p.group + g;
          const __nv_bfloat16* src = p.q + row * D;
          if (kQ4) {   // the places of a code word's dims
            const __nv_bfloat16* w = src + (piece >> 2) * 32 + (piece & 3) * 4;
            a[i] = *reinterpret_cast<const uint2*>(w);
            b[i] = *reinterpret_cast<const uint2*>(w + 16);
          } else {
            const uint4 v = *reinterpret_cast<const uint4*>(src + piece * 8);
            a[i] = make_uint2(v.x, v.y);
            b[i] = make_uint2(v.z, v.w);
          }
          l[i] = p.lse[row];
        }
        // the last run's products have read theirs
        if (rb == 0 && ok && run > 0)
          ok = __all_sync(0xFFFFFFFFu, role_wait(&b_qfree, (run - 1) & 1, &s_dead));
        if (!ok) break;
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const int r = rb + i * kPerStep + warp * (32 / kLanes) + lane / kLanes;
          if (rb + i * kPerStep >= R) break;
          uint32_t m = __vmaxu2(__vmaxu2(a[i].x & 0x7FFF7FFFu, a[i].y & 0x7FFF7FFFu),
                                __vmaxu2(b[i].x & 0x7FFF7FFFu, b[i].y & 0x7FFF7FFFu));
          m = max(m & 0xFFFFu, m >> 16);
#pragma unroll
          for (int o = kLanes / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
          // a row that is not finite counts for nothing
          const bool fine = s[i] >= 0 && m < 0x7F80u && fabsf(l[i]) < INFINITY;
          if (bad[i]) problems |= DFV_DEV_BAD_PATH;
          if (s[i] >= 0 && !fine) problems |= DFV_DEV_NONFINITE;
          a[i] = fine ? a[i] : make_uint2(0, 0);
          b[i] = fine ? b[i] : make_uint2(0, 0);
          const float off = fine ? -l[i] * 1.44269504f : -INFINITY;
          const int last = fine ? at0 + s[i] : -1;
          const int first = p.window > 0 ? last - p.window + 1 : 0;
          int e = max(fine ? static_cast<int>(m >> 7) : 0, 40);   // all below 2^(e - 126)
          if (!kBlocks) {
            if (!fine || (e <= e_tile && e >= e_tile - 8)) e = e_tile;
            else own = true;
          }
          const float f = pow2i(141 - e);                               // to below 2^15
          const float slope = p.scale * 1.44269504f * pow2i(e - 141);
          if (r < R) {
            auto half2_of = [](uint32_t lo16, uint32_t hi16, float f) {
              return pack_half2(__uint_as_float(lo16 << 16) * f, __uint_as_float(hi16 << 16) * f);
            };
            const float g = kBlocks ? f * 0.0625f : f;   // high nibbles are 16 times as large
            const uint2 x = a[i], y = b[i];
            uint4 o;
            if (kQ4)   // dims {0, 2, 16, 18, 1, 3, 17, 19} of the word
              o = make_uint4(half2_of(x.x & 0xFFFFu, x.y & 0xFFFFu, f),
                             half2_of(y.x & 0xFFFFu, y.y & 0xFFFFu, g),
                             half2_of(x.x >> 16, x.y >> 16, f), half2_of(y.x >> 16, y.y >> 16, g));
            else
              o = make_uint4(half2_of(x.x & 0xFFFFu, x.x >> 16, f),
                             half2_of(x.y & 0xFFFFu, x.y >> 16, f),
                             half2_of(y.x & 0xFFFFu, y.x >> 16, f),
                             half2_of(y.y & 0xFFFFu, y.y >> 16, f));
            *reinterpret_cast<uint4*>(sQ + tc::sw128_offset(r, piece, R)) = o;
            if (piece == 0) {
              s_slope[tb][r] = slope;
              s_off[tb][r] = off;
              s_first[tb][r] = first;
              s_last[tb][r] = last;
            }
          }
        }
      }
      if (problems) report(p.status, problems);
      fence_proxy_async_smem();
      __syncwarp();
      if (ok && lane == 0) mbar_arrive(&b_q);
      // The columns' factors are everyone's. All eight warps come here in every
      // run, whatever their waits gave, and end together.
      ok = named_sync_and(1, 256, ok);
      if (!ok) return false;
      const bool same = kBlocks || named_sync_and(1, 256, !own);
      const float slope_all = p.scale * 1.44269504f * pow2i(e_tile - 141);
      const float* slope = s_slope[tb];
      const float* off = s_off[tb];
      for (int c = c0; ok && c < c1; ++c, ++k) {
        if ((k & 1) != grp) continue;
        const int j = c * kWtKeys + (warp & 3) * 32 + lane;
        float* dst = p.weights + static_cast<int64_t>(h) * p.capacity + j;
        float had = 0.0f;
        if (j < C) {
          if (t > 0) had = *dst;
          else if (p.prev && j < at0)
            had = p.decay * p.prev[static_cast<int64_t>(h) * p.capacity + j];
        }
        // every row sees the whole chunk: up to row 0's own place, from the last row's window on
        const bool whole = (c + 1) * kWtKeys <= at0 + 1 &&
                           (p.window == 0 || c * kWtKeys >= C - p.window);
        float s0 = 0.0f, s1 = 0.0f, s2 = 0.0f, s3 = 0.0f;
        uint32_t ts = 0;   // column 0 of the tile, were the slice's neighbours beside it
        auto add = [&](auto columns, auto plain, int r) {
          constexpr int kN = decltype(columns)::value;
          constexpr bool kPlain = decltype(plain)::value != 0;
          uint32_t x[kN];
          if constexpr (kBlocks) {
            // the blocks' sums times this key's scales, two blocks at a time
            const int key = (warp & 3) * 32 + lane;
#pragma unroll
            for (int i = 0; i < D / 64; ++i) {
              uint32_t z[32];
              tc::TmemIo<32>::load(ts + i * 32, z);
              const float d0 = __half2float(s_scale[k & 3][2 * i][key]);
              const float d1 = __half2float(s_scale[k & 3][2 * i + 1][key]);
#pragma unroll
              for (int e = 0; e < 16; e += 2) {
                float a = i == 0 ? 0.0f : __uint_as_float(x[e]);
                float b = i == 0 ? 0.0f : __uint_as_float(x[e + 1]);
                fma2(a, b, __uint_as_float(z[e]), __uint_as_float(z[e + 1]), d0, d0, a, b);
                fma2(a, b, __uint_as_float(z[16 + e]), __uint_as_float(z[16 + e + 1]), d1, d1, a, b);
                x[e] = __float_as_uint(a);
                x[e + 1] = __float_as_uint(b);
              }
            }
          } else {
            tc::TmemIo<kN>::load(ts + r, x);
          }
#pragma unroll
          for (int i = 0; i < kN; i += 4) {
            const float4 f = kPlain && !kBlocks
                                 ? make_float4(slope_all, slope_all, slope_all, slope_all)
                                 : *reinterpret_cast<const float4*>(slope + r + i);
            const float4 o = *reinterpret_cast<const float4*>(off + r + i);
            float y0, y1, y2, y3;
            fma2(y0, y1, __uint_as_float(x[i]), __uint_as_float(x[i + 1]), f.x, f.y, o.x, o.y);
            fma2(y2, y3, __uint_as_float(x[i + 2]), __uint_as_float(x[i + 3]), f.z, f.w, o.z, o.w);
            y0 = tc::ex2(y0), y1 = tc::ex2(y1), y2 = tc::ex2(y2), y3 = tc::ex2(y3);
            if constexpr (!kPlain) {
              const int4 a = *reinterpret_cast<const int4*>(s_first[tb] + r + i);
              const int4 b = *reinterpret_cast<const int4*>(s_last[tb] + r + i);
              y0 = j >= a.x && j <= b.x ? y0 : 0.0f;
              y1 = j >= a.y && j <= b.y ? y1 : 0.0f;
              y2 = j >= a.z && j <= b.z ? y2 : 0.0f;
              y3 = j >= a.w && j <= b.w ? y3 : 0.0f;
            }
            add2(s0, s1, s0, s1, y0, y1);
            add2(s2, s3, s2, s3, y2, y3);
          }
        };
        for (int sl = 0; ok && sl < slices; ++sl) {
          ok = __all_sync(0xFFFFFFFFu, role_wait(&b_s[place], turn & 1, &s_dead));
          if (!ok) break;
          tc::fence_after_sync();
          ts = tmem + lanes + W::kTS + place * place_cols - sl * RS;
          auto add_all = [&](auto plain) {
            int r = sl * RS;
            const int end = r + RS;
            if constexpr (!kBlocks)
              for (; r + 32 <= end; r += 32) add(Columns<32>(), plain, r);
            if (r < end) add(Columns<16>(), plain, r);
          };
          // (the same rows: 57 us, with the test of `whole` within the loop 73)
          if (whole && same) add_all(Columns<1>());
          else add_all(Columns<0>());
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(&b_sfree[place]);
          if constexpr (kSliced) skip(place, turn, 1);
        }
        if constexpr (kSliced) skip(place, turn, slices);   // the other group's
        else ++turn;
        if (!ok) break;
        if (j < C) *dst = had + ((s0 + s1) + (s2 + s3));
      }
      ++run;
      return true;
    });
    // keys that no row sees keep what they had
    if (ok) {
      const int seen = min(C, fc * kWtKeys), rest = tiles == 0 ? C : seen;
      const int64_t total = static_cast<int64_t>(p.hkv) * rest;
      for (int64_t i = blockIdx.x * 256 + tid; i < total;
           i += static_cast<int64_t>(gridDim.x) * 256) {
        const int64_t h = i / rest, j = i - h * rest;
        const int64_t at = h * p.capacity + j;
        p.weights[at] = p.prev && j < at0 ? p.decay * p.prev[at] : 0.0f;
      }
    }
    tc::fence_before_sync();
  }
  __syncwarp();
  __syncthreads();
  if (warp == kWtMma) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, 512);
  }
  if (tid == 0 && s_dead) report(p.status, DFV_DEV_TIMEOUT);
}

template <int D, int kMode>
dfv_status weights_launch(const WeightParams& p, cudaStream_t stream) {
  using W = WeightShape<D, kMode>;
  static std::atomic<int> allowed[64];   // per device
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return DFV_ERR_CUDA;
  if (!allowed[dev].load(std::memory_order_acquire)) {
    if (cudaFuncSetAttribute(kv_weights_kernel<D, kMode>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                             W::kBytes) != cudaSuccess)
      return DFV_ERR_CUDA;
    allowed[dev].store(1, std::memory_order_release);
  }
  const int64_t most =
      static_cast<int64_t>(p.hkv) * ((static_cast<int64_t>(p.capacity) + kWtKeys - 1) / kWtKeys);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(most < sm_count() ? most : sm_count()));
  cfg.blockDim = dim3(kWtThreads);
  cfg.dynamicSmemBytes = W::kBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv_weights_kernel<D, kMode>, p) == cudaSuccess ? DFV_OK
                                                                               : DFV_ERR_CUDA;
}

template <int D>
dfv_status weights_launch_f(const WeightParams& p, bool q4, cudaStream_t stream) {
  const int64_t rows = static_cast<int64_t>(p.n_rows) * p.group;
  if (q4)
    return rows <= WeightShape<D, kModeBlocks>::kRows ? weights_launch<D, kModeBlocks>(p, stream)
                                                      : weights_launch<D, kModeSplit>(p, stream);
  if constexpr (D < 256)
    if (rows > WeightShape<D, kModeF16>::kRows) return weights_launch<D, kModeSliced>(p, stream);
  return weights_launch<D, kModeF16>(p, stream);
}

}  // namespace dfv

extern "C" dfv_status dfv_kv_weights(int n_rows, int n_q_heads, int n_kv_heads, int head_dim,
                                     int window, int kv_format, int cache_capacity,
                                     const int32_t* ctx_len, const void* k_cache, const void* q,
                                     const float* lse, const int32_t* path,
                                     const int32_t* accept_len, float scale, float decay,
                                     const float* prev, float* weights, uint32_t* status,
                                     dfv_stream_t stream) {
  using namespace dfv;
  if ((kv_format != DFV_KV_Q4_0 && kv_format != DFV_KV_F16) ||
      (head_dim != 64 && head_dim != 128 && head_dim != 256))
    return DFV_ERR_UNSUPPORTED;
  if (n_rows < 1 || n_rows > 65536 || n_kv_heads < 1 || n_q_heads < n_kv_heads ||
      n_q_heads > 1024 || n_q_heads % n_kv_heads != 0 || window < 0 || cache_capacity < 1 ||
      cache_capacity > (1 << 30) || scale != scale || decay != decay)
    return DFV_ERR_INVALID;
  if (!ctx_len || !k_cache || !q || !lse || !weights || !aligned(k_cache, 16) ||
      !aligned(q, 16) || !aligned(lse, 4) || !aligned(prev, 4) || !aligned(weights, 4) ||
      !aligned(ctx_len, 4) || !aligned(path, 4) || !aligned(accept_len, 4))
    return DFV_ERR_INVALID;
  if (scale <= 0.0f) scale = head_dim == 64 ? 0.125f : head_dim == 256 ? 0.0625f : 0.08838834765f;
  if (window >= cache_capacity) window = 0;   // (hides nothing; and no difference overflows)
  const uint32_t group = static_cast<uint32_t>(n_q_heads / n_kv_heads);
  // (exact while rows * group stays below 2^32)
  const uint32_t group_m =
      group == 1 || static_cast<uint64_t>(n_rows) * group * group >= 1ull << 32
          ? 0u
          : static_cast<uint32_t>(((1ull << 32) + group - 1) / group);
  const WeightParams p = {n_rows, n_q_heads, n_kv_heads, n_q_heads / n_kv_heads, window,
                          cache_capacity, group_m, ctx_len, static_cast<const uint8_t*>(k_cache),
                          static_cast<const __nv_bfloat16*>(q), lse, path, accept_len, scale,
                          decay, prev, weights, status};
  const bool q4 = kv_format == DFV_KV_Q4_0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return head_dim == 64    ? weights_launch_f<64>(p, q4, s)
         : head_dim == 128 ? weights_launch_f<128>(p, q4, s)
                           : weights_launch_f<256>(p, q4, s);
}
