// Writing the 8-bit cache (rows appended, accepted rows committed) and
// reading it back.
//
// A block is quantised once, when its 64 positions are complete, from their
// bf16 values:
//
//   amax = max |x| over the block's 64 * D values,  scale = amax / 127,
//   code = round-half-even(127 x / amax)
//
// so the cache's content does not depend on how the rows arrived (one prompt,
// single tokens, accepted rows of a tree). 127 x is exact in f32 for a bf16
// x, and one correctly rounded division of it cannot turn a quotient that is
// no tie into a tie or the reverse (with 8-bit significands a quotient that
// misses a half-way point misses it by 2^-17 at least), so the rule is the
// exact rounding of the real quotient. The kernel multiplies by 127 / amax
// (an error below 2^-15) and divides only where the product is that near to
// a half-way point.
//
// Both kernels are bound by memory: 2 (4 for f32) bytes in and 1 out a value,
// 1 in and 2 (4) out. One CTA of D threads takes one block of K or V of one
// head, 64 values a thread in registers, so every value is read once and the
// block's maximum needs no second pass. A K thread holds four pieces of 16
// dims of one position, a V thread 4 dims of 16 positions: the piece of the
// layout that it writes is then whole in its registers.

#include <atomic>

#include "kv8.cuh"

namespace dfv {

struct Kv8AppendParams {
  dfv_kv8_cache c;
  int nblk;            // blocks a head has room for
  int at, n;           // at < 0: the committed length
  const void* src[2];
  int64_t s_row[2], s_head[2];
  const int32_t* path;        // with accept_len: row k of the write is src row path[k]
  const int32_t* accept_len;
  int n_nodes;
  int bulk;      // blocks b0 + 1 .. b0 + bulk are written by kv8_append_bulk_kernel
  uint32_t* status;
};

// The rows of a write, agreed on by every CTA.
struct Kv8Span {
  int at, end;     // positions written
  int b0, open;    // first block touched, block that is open afterwards
};

__device__ __forceinline__ uint32_t bf16x2_bits(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// 32 bytes in one access; the address is a multiple of 32.
__device__ __forceinline__ void ld32b(const void* p, uint32_t* w) {
  asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]),
                 "=r"(w[6]), "=r"(w[7])
               : "l"(p)
               : "memory");
}
__device__ __forceinline__ void st32b(void* p, const uint32_t* w) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]),
               "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// kN (4 or 16) values from global memory as packed bf16 (f32: rounded to
// nearest even).
template <typename T, int kN, bool kVec>
__device__ __forceinline__ void load_bf16(const T* s, uint32_t* w) {
  if constexpr (!kVec) {
#pragma unroll
    for (int k = 0; k < kN / 2; ++k) {
      if constexpr (sizeof(T) == 4) {
        w[k] = bf16x2_bits(s[2 * k], s[2 * k + 1]);
      } else {
        const uint16_t* u = reinterpret_cast<const uint16_t*>(s);
        w[k] = u[2 * k] | (static_cast<uint32_t>(u[2 * k + 1]) << 16);
      }
    }
  } else if constexpr (sizeof(T) == 4) {
    if constexpr (kN == 16) {
      uint32_t f[16];
      ld32b(s, f);
      ld32b(s + 8, f + 8);
#pragma unroll
      for (int k = 0; k < 8; ++k)
        w[k] = bf16x2_bits(__uint_as_float(f[2 * k]), __uint_as_float(f[2 * k + 1]));
    } else {
      const float4 v = *reinterpret_cast<const float4*>(s);
      w[0] = bf16x2_bits(v.x, v.y);
      w[1] = bf16x2_bits(v.z, v.w);
    }
  } else if constexpr (kN == 16) {
    ld32b(s, w);
  } else {
    const uint2 v = *reinterpret_cast<const uint2*>(s);
    w[0] = v.x;
    w[1] = v.y;
  }
}

// Four values as codes, lowest byte first. Adding 1.5 * 2^23 rounds to the
// nearest even integer and leaves it in the low bits.
__device__ __forceinline__ uint32_t quantise4(float a, float b, float c, float d, float inv,
                                              float amax) {
  constexpr float kMagic = 12582912.0f;
  const float x[4] = {a, b, c, d};
  float r[4], off = 0.0f;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float t = x[k] * inv;
    r[k] = t + kMagic;
    off = fmaxf(off, fabsf(t - (r[k] - kMagic)));
  }
  if (off > 0.4998f) {   // near a half-way point: by the exact quotient
#pragma unroll
    for (int k = 0; k < 4; ++k) r[k] = __fdiv_rn(x[k] * 127.0f, amax) + kMagic;
  }
  const uint32_t lo = __byte_perm(__float_as_uint(r[0]), __float_as_uint(r[1]), 0x0040);
  const uint32_t hi = __byte_perm(__float_as_uint(r[2]), __float_as_uint(r[3]), 0x0040);
  return __byte_perm(lo, hi, 0x5410);
}

// The 64 values of one thread: 32 packed words. K: piece j of 16 dims at w[8 j]; V: position i of
// 16 at w[2 i].
template <typename T, int D, bool kVec>
struct BlockIo {
  static constexpr int kTpt = D / 64;      // K: threads per position
  static constexpr int kVt = D / 4;        // V: threads per 16 positions

  // Piece `dim` (kN values) of the rows pos + 0 .. kRows - 1, row i at
  // w[i * kN / 2]: source rows, tail rows where the block is complete and
  // begins before the write, zeros elsewhere. Every load is issued whatever
  // the row (from a row that exists) and the choice made on its value: a
  // branch per row would wait for each load in turn.
  template <bool kV, int kN, int kRows>
  static __device__ __forceinline__ void load_rows(const Kv8AppendParams& p, const Kv8Span& s,
                                                   const int* path, int h, int b, int pos,
                                                   int dim, uint32_t* w) {
    const int n = s.end - s.at;
    if (n > 0) {
      const T* src = static_cast<const T*>(p.src[kV]) + h * p.s_head[kV] + dim;
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const int k = min(max(pos + i - s.at, 0), n - 1);
        load_bf16<T, kN, kVec>(src + (path ? path[k] : k) * p.s_row[kV], w + i * kN / 2);
      }
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i)
      if (pos + i < s.at || pos + i >= s.end) {
#pragma unroll
        for (int e = 0; e < kN / 2; ++e) w[i * kN / 2 + e] = 0u;
      }
    if (s.at <= b * kBlk || s.end < (b + 1) * kBlk) return;
    const __nv_bfloat16* tail = static_cast<const __nv_bfloat16*>(kV ? p.c.v_tail : p.c.k_tail) +
                                (static_cast<int64_t>(h) * 2 + (b & 1)) * kBlk * D + dim;
    uint32_t t[kN / 2 * kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i)
      load_bf16<__nv_bfloat16, kN, true>(tail + min(pos + i, s.at - 1) % kBlk * D, t + i * kN / 2);
#pragma unroll
    for (int i = 0; i < kRows; ++i)
      if (pos + i < s.at) {
#pragma unroll
        for (int e = 0; e < kN / 2; ++e) w[i * kN / 2 + e] = t[i * kN / 2 + e];
      }
  }

  template <bool kV>
  static __device__ __forceinline__ void load(const Kv8AppendParams& p, const Kv8Span& s,
                                              const int* path, int h, int b, uint32_t* w) {
    const int tid = threadIdx.x;
    if (!path && b * kBlk >= s.at && (b + 1) * kBlk <= s.end) {   // source rows throughout
      const T* src = static_cast<const T*>(p.src[kV]) + h * p.s_head[kV];
      const int64_t r0 = b * kBlk - s.at;
      if constexpr (!kV) {
        src += (r0 + tid / kTpt) * p.s_row[0] + tid % kTpt * 16;
#pragma unroll
        for (int j = 0; j < 4; ++j) load_bf16<T, 16, kVec>(src + j * kTpt * 16, w + 8 * j);
      } else {
        src += (r0 + tid / kVt * 16) * p.s_row[1] + tid % kVt * 4;
#pragma unroll
        for (int i = 0; i < 16; ++i) load_bf16<T, 4, kVec>(src + i * p.s_row[1], w + 2 * i);
      }
    } else if constexpr (!kV) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        load_rows<false, 16, 1>(p, s, path, h, b, b * kBlk + tid / kTpt,
                                (tid % kTpt + j * kTpt) * 16, w + 8 * j);
    } else {
      load_rows<true, 4, 16>(p, s, path, h, b, b * kBlk + tid / kVt * 16, tid % kVt * 4, w);
    }
  }

  // Rows of block b written by this call, into their tail slot.
  template <bool kV>
  static __device__ __forceinline__ void store_tail(const Kv8AppendParams& p, const Kv8Span& s,
                                                    int h, int b, const uint32_t* w) {
    const int tid = threadIdx.x;
    __nv_bfloat16* slot = static_cast<__nv_bfloat16*>(kV ? p.c.v_tail : p.c.k_tail) +
                          (static_cast<int64_t>(h) * 2 + (b & 1)) * kBlk * D;
    if constexpr (!kV) {
      const int t = tid / kTpt, pos = b * kBlk + t;
      if (pos < s.at || pos >= s.end) return;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint4* dst = reinterpret_cast<uint4*>(slot + t * D + (tid % kTpt + j * kTpt) * 16);
        dst[0] = make_uint4(w[8 * j], w[8 * j + 1], w[8 * j + 2], w[8 * j + 3]);
        dst[1] = make_uint4(w[8 * j + 4], w[8 * j + 5], w[8 * j + 6], w[8 * j + 7]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int t = tid / kVt * 16 + i, pos = b * kBlk + t;
        if (pos >= s.at && pos < s.end)
          *reinterpret_cast<uint2*>(slot + t * D + tid % kVt * 4) =
              make_uint2(w[2 * i], w[2 * i + 1]);
      }
    }
  }

  template <bool kV>
  static __device__ __forceinline__ void store_codes(const Kv8AppendParams& p, int h, int b,
                                                     const uint32_t* w, uint32_t amax_bits) {
    const int tid = threadIdx.x;
    const bool zero = amax_bits < kSmallBits;
    const float amax = __uint_as_float(amax_bits << 16);
    const float inv = zero ? 0.0f : __fdiv_rn(127.0f, amax);
    if (tid == 0)
      (kV ? p.c.v_scale : p.c.k_scale)[static_cast<int64_t>(h) * p.nblk + b] =
          zero ? 0.0f : __fdiv_rn(amax, 127.0f);
    int8_t* base = (kV ? p.c.v_codes : p.c.k_codes) + static_cast<int64_t>(h) * p.nblk * kBlk * D;
    if constexpr (!kV) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t q[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t a = w[8 * j + 2 * e], c = w[8 * j + 2 * e + 1];
          q[e] = quantise4(bf16_lo(a), bf16_hi(a), bf16_lo(c), bf16_hi(c), inv, amax);
        }
        *reinterpret_cast<uint4*>(base + kv8_k_piece(b, tid / kTpt, tid % kTpt + j * kTpt, D)) =
            make_uint4(q[0], q[1], q[2], q[3]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; j += 2) {   // two of the thread's dims: 32 bytes in a row
        uint32_t q[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float x[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t a = w[2 * (4 * (e & 3) + i) + j / 2];
            x[i] = e >= 4 ? bf16_hi(a) : bf16_lo(a);
          }
          q[e] = quantise4(x[0], x[1], x[2], x[3], inv, amax);
        }
        st32b(base + kv8_v_piece(b, tid / kVt, tid % kVt * 4 + j, D), q);
      }
    }
  }
};

// Largest magnitude of a thread's values (bf16 bits).
__device__ __forceinline__ uint32_t max_bits(const uint32_t* w) {
  uint32_t m = 0;
#pragma unroll
  for (int k = 0; k < 32; ++k) m = __vmaxu2(m, w[k] & 0x7FFF7FFFu);
  return max(m & 0xFFFFu, m >> 16);
}

// The same once values that are not stored have become zeros.
__device__ __forceinline__ uint32_t keep_storable(uint32_t* w, uint32_t* status) {
  const uint32_t m = max_bits(w);
  if (m < kBigBits) return m;
  report(status, DFV_DEV_NONFINITE);
#pragma unroll
  for (int k = 0; k < 32; ++k) {
    if ((w[k] & 0x7FFFu) >= kBigBits) w[k] &= 0xFFFF0000u;
    if (((w[k] >> 16) & 0x7FFFu) >= kBigBits) w[k] &= 0x0000FFFFu;
  }
  return max_bits(w);
}

// The block of this CTA. `refused` is asked once the block's loads are in
// flight; nothing is written if it says so. True if the CTA is the last of
// the grid to have read the cache's state.
template <typename T, int D, bool kVec, bool kV, typename F>
__device__ __forceinline__ bool append_block(const Kv8AppendParams& p, const Kv8Span& s,
                                             const int* path, uint32_t* s_max, F refused) {
  using Io = BlockIo<T, D, kVec>;
  const int h = blockIdx.y;
  const int b = s.b0 + static_cast<int>(blockIdx.x) + (blockIdx.x > 0 ? p.bulk : 0);
  const int tid = threadIdx.x;
  const bool mine = b * kBlk < s.end;
  uint32_t w[32];
  if (mine) Io::template load<kV>(p, s, path, h, b, w);
  if (refused()) return false;
  uint32_t m = 0;
  if (mine) m = __reduce_max_sync(0xFFFFFFFFu, keep_storable(w, p.status));
  if ((tid & 31) == 0) s_max[tid >> 5] = m;
  __syncthreads();   // also: the block's tail rows and the state have been read
  unsigned ticket = 0;
  if (tid == 0) ticket = atomicAdd(reinterpret_cast<unsigned*>(p.c.state) + 1, 1u);
  if (mine) {
#pragma unroll
    for (int k = 0; k < D / 32; ++k) m = max(m, s_max[k]);
    if (s.end >= (b + 1) * kBlk) Io::template store_codes<kV>(p, h, b, w, m);
    // The blocks that the tail keeps afterwards are the open one and the one
    // before. Their slots may hold rows that block b0 still needs (its own
    // slot has the same parity every second block); b0's CTA then writes them.
    const bool shared = s.at % kBlk != 0;   // b0 reads its slot
    if (b >= s.open - 1 && (b == s.b0 || !shared || ((b - s.b0) & 1)))
      Io::template store_tail<kV>(p, s, h, b, w);
    if (b == s.b0 && shared) {
      const int other = ((s.open - s.b0) & 1) ? s.open - 1 : s.open;
      if (other > b) {
        Io::template load<kV>(p, s, path, h, other, w);
        keep_storable(w, p.status);
        Io::template store_tail<kV>(p, s, h, other, w);
      }
    }
  }
  return tid == 0 && ticket == gridDim.x * gridDim.y * gridDim.z - 1;
}

template <typename T, int D, bool kVec>
__global__ void __launch_bounds__(D) kv8_append_kernel(const __grid_constant__ Kv8AppendParams p) {
  __shared__ uint32_t s_max[D / 32];
  __shared__ int s_path[kMaxNodes];
  __shared__ int s_bad;
  const int tid = threadIdx.x;
  grid_dep_wait();
  grid_dep_launch_dependents();   // (after the wait: see common.cuh)
  const int C = static_cast<volatile int32_t*>(p.c.state)[0];
  const int held = static_cast<volatile int32_t*>(p.c.state)[2];
  const int stopped = static_cast<volatile int32_t*>(p.c.state)[3];
  int at = p.at, n = p.n;
  uint32_t bad = stopped ? DFV_DEV_TIMEOUT : 0;   // a wait of a long write gave up
  if (at < 0) {
    if (C < 0 || C > p.c.capacity) bad |= DFV_DEV_CTX;
    at = C;
  }
  if (p.accept_len) {
    n = *p.accept_len;
    if (n < 1 || n > p.n_nodes) bad |= DFV_DEV_BAD_PATH;
    if (tid == 0) s_bad = 0;
    __syncthreads();
    if (!bad)
      for (int k = tid; k < n; k += D) {
        const int node = p.path[k];
        s_path[k] = node;
        if (node < 0 || node >= p.n_nodes) s_bad = 1;
      }
    __syncthreads();
    if (s_bad) bad |= DFV_DEV_BAD_PATH;
  }
  if (!bad && n > p.c.capacity - at) bad = DFV_DEV_CAPACITY;   // (no sum: both reach 2^30)
  // the rows of at's block before it have to be in the tail
  auto refused = [&]() {
    if (C < 0 || C > p.c.capacity || at > C || (at % kBlk != 0 && at / kBlk < held))
      bad |= DFV_DEV_CTX;
    if (bad && tid == 0 && blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0)
      report(p.status, bad);
    return bad != 0;   // the same for every CTA: nothing is written
  };
  if (bad) {
    refused();
    return;
  }
  Kv8Span s;
  s.at = at;
  s.end = at + n;
  s.b0 = at / kBlk;
  s.open = s.end / kBlk;
  const int* path = p.accept_len ? s_path : nullptr;
  const bool last = blockIdx.z == 0
                        ? append_block<T, D, kVec, false>(p, s, path, s_max, refused)
                        : append_block<T, D, kVec, true>(p, s, path, s_max, refused);
  // The last CTA to have read the state advances the committed length; the
  // counter beside it is left at zero. (What the grid writes is read by later
  // launches only.)
  if (last) {
    p.c.state[1] = 0;
    p.c.state[0] = s.end;
    // the first block whose bf16 rows the tail now has
    p.c.state[2] = s.open > s.b0 ? s.open - 1 : s.b0 < held ? s.b0 : max(held, s.b0 - 1);
  }
}

// The inner blocks of a long write of bf16 rows: source rows throughout, and
// none that the tail keeps. One wave of CTAs walks over them while the copy
// engine brings each CTA its next block: with loads to registers a CTA's loads
// and its arithmetic took turns (61440 rows of 4 heads of 256, written and
// read back: 151 us, here 140; three slots and two CTAs an SM: 165). The
// launch before kv8_append_kernel, which takes the blocks at both ends and
// advances the length.
constexpr int kBulkSlots = 2;

template <int D>
__global__ void __launch_bounds__(D)
    kv8_append_bulk_kernel(const __grid_constant__ Kv8AppendParams p) {
  using Io = BlockIo<__nv_bfloat16, D, true>;
  constexpr int kSlot = kBlk * D * 2;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t full[kBulkSlots];
  __shared__ uint32_t s_max[2][D / 32];
  __shared__ int s_stopped;
  constexpr uint32_t kNoRows = ~0u;   // in a maximum's place: a thread's wait gave up
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    for (int k = 0; k < kBulkSlots; ++k) mbar_init(&full[k], 1);
    fence_mbar_init();
  }
  grid_dep_wait();
  const int C = p.c.state[0], held = p.c.state[2];
  const int at = p.at < 0 ? C : p.at;
  // (asked by one thread: another CTA of this launch may set it meanwhile)
  if (tid == 0) s_stopped = static_cast<volatile int32_t*>(p.c.state)[3];
  __syncthreads();
  // refused as by kv8_append_kernel, which reports it
  if (s_stopped != 0 || C < 0 || C > p.c.capacity || at > C || p.n > p.c.capacity - at ||
      (at % kBlk != 0 && at / kBlk < held))
    return;
  fence_proxy_async_global();   // what earlier kernels wrote, to the copy engine
  const int b0 = at / kBlk, per = p.bulk * p.c.n_kv_heads;   // blocks of K, as many of V
  const int total = 2 * per;
  // block `it` of the walk, a head's blocks in a row
  auto copy = [&](int it, int slot) {
    const int kv = it >= per, r = kv ? it - per : it;
    const int h = r / p.bulk, b = b0 + 1 + r - h * p.bulk;
    const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(p.src[kv]) + h * p.s_head[kv] +
                               static_cast<int64_t>(b * kBlk - at) * p.s_row[kv];
    if (lane == 0) mbar_arrive_expect_tx(&full[slot], kSlot);
    __syncwarp();
    for (int t = lane; t < kBlk; t += 32)
      bulk_g2s(smem + slot * kSlot + t * D * 2, src + t * p.s_row[kv], D * 2, &full[slot]);
  };
  const int step = gridDim.x;
  int it = blockIdx.x;
  if (warp == 0)
    for (int k = 0; k < kBulkSlots - 1; ++k)
      if (it + k * step < total) copy(it + k * step, k);
  int k = 0;
  for (; it < total; it += step, ++k) {
    const int slot = k % kBulkSlots;
    // the slot freed by the last block's reads (a barrier ago) is filled again
    if (warp == 0 && it + (kBulkSlots - 1) * step < total)
      copy(it + (kBulkSlots - 1) * step, (k + kBulkSlots - 1) % kBulkSlots);
    const bool there = mbar_wait_bounded(&full[slot], (k / kBulkSlots) & 1);
    const int kv = it >= per, r = kv ? it - per : it;
    const int h = r / p.bulk, b = b0 + 1 + r - h * p.bulk;
    const uint8_t* rows = smem + slot * kSlot;
    uint32_t w[32];
    if (kv == 0) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint4* s = reinterpret_cast<const uint4*>(
            rows + tid / Io::kTpt * D * 2 + (tid % Io::kTpt + j * Io::kTpt) * 32);
        *reinterpret_cast<uint4*>(w + 8 * j) = s[0];
        *reinterpret_cast<uint4*>(w + 8 * j + 4) = s[1];
      }
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const uint2 v = *reinterpret_cast<const uint2*>(
            rows + (tid / Io::kVt * 16 + i) * D * 2 + tid % Io::kVt * 8);
        w[2 * i] = v.x;
        w[2 * i + 1] = v.y;
      }
    }
    uint32_t m = __reduce_max_sync(0xFFFFFFFFu, there ? keep_storable(w, p.status) : kNoRows);
    if (lane == 0) s_max[k & 1][warp] = m;
    __syncthreads();   // maxima are there, and the slot has been read
#pragma unroll
    for (int e = 0; e < D / 32; ++e) m = max(m, s_max[k & 1][e]);
    if (m == kNoRows) break;   // nothing is stored of rows that did not come
    if (kv == 0) Io::template store_codes<false>(p, h, b, w, m);
    else Io::template store_codes<true>(p, h, b, w, m);
  }
  if (it < total && tid == 0) {
    // No later write advances the length over what is missing: kv8_append_kernel
    // asks for this word. Copies in flight land before the CTA ends.
    *static_cast<volatile int32_t*>(p.c.state + 3) = 1;
    report(p.status, DFV_DEV_TIMEOUT);
    for (int j = 0; j < kBulkSlots; ++j)
      if (it + j * step < total)
        mbar_wait_bounded(&full[(k + j) % kBulkSlots], ((k + j) / kBulkSlots) & 1);
  }
  // Not earlier: CTAs of the launches behind, waiting in an SM's room, would
  // keep some of the next write's wave out (six caches in turn, 61440 rows of
  // 4 heads of 256 each: 132 us a write, so 92).
  grid_dep_launch_dependents();
}

// Launch that may be set up while the kernel before it runs (its kernels wait
// for that one before they touch anything).
template <typename P>
dfv_status launch_after(void (*kernel)(P), dim3 grid, int threads, const P& p,
                        cudaStream_t stream, int smem = 0) {
  cudaLaunchConfig_t cfg = {};
  cfg.dynamicSmemBytes = smem;
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p) == cudaSuccess ? DFV_OK : DFV_ERR_CUDA;
}

template <int D>
dfv_status bulk_launch(const Kv8AppendParams& p, cudaStream_t stream) {
  constexpr int kSmem = kBulkSlots * kBlk * D * 2;
  static std::atomic<int> configured[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return DFV_ERR_CUDA;
  if (!configured[dev].load(std::memory_order_acquire)) {
    if (cudaFuncSetAttribute(kv8_append_bulk_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kSmem) != cudaSuccess)
      return DFV_ERR_CUDA;
    configured[dev].store(1, std::memory_order_release);
  }
  const int most = sm_count() * (768 / D);   // 64 KB of slots and 256 threads, three times an SM
  const int64_t blocks = 2ll * p.bulk * p.c.n_kv_heads;
  return launch_after(kv8_append_bulk_kernel<D>, dim3(blocks < most ? blocks : most), D, p, stream,
                      kSmem);
}

template <typename T, bool kVec>
dfv_status append_launch_t(Kv8AppendParams& p, int rows, cudaStream_t stream) {
  int blocks = (rows + kBlk - 2) / kBlk + 1;   // that `rows` can touch
  if constexpr (sizeof(T) == 2 && kVec) {
    // Wherever the write starts, blocks b0 + 1 .. b0 + n / 64 - 2 are complete
    // and not among the two that the tail keeps. Worth a launch of their own
    // from about four waves of blocks on.
    const int inner = p.accept_len ? 0 : rows / kBlk - 2;
    if (static_cast<int64_t>(inner) * p.c.n_kv_heads * p.c.head_dim >= 512ll * 2 * sm_count()) {
      p.bulk = inner;
      blocks -= inner;
      const dfv_status st = p.c.head_dim == 64    ? bulk_launch<64>(p, stream)
                            : p.c.head_dim == 128 ? bulk_launch<128>(p, stream)
                                                  : bulk_launch<256>(p, stream);
      if (st != DFV_OK) return st;
    }
  }
  const dim3 grid(blocks, p.c.n_kv_heads, 2);
  switch (p.c.head_dim) {
    case 64: return launch_after(kv8_append_kernel<T, 64, kVec>, grid, 64, p, stream);
    case 128: return launch_after(kv8_append_kernel<T, 128, kVec>, grid, 128, p, stream);
    default: return launch_after(kv8_append_kernel<T, 256, kVec>, grid, 256, p, stream);
  }
}

dfv_status kv8_append_launch(Kv8AppendParams& p, int rows, int dtype, cudaStream_t stream) {
  p.nblk = kv8_blocks(p.c.capacity);
  const int e = dtype == DFV_DTYPE_F32 ? 4 : 2;
  bool vec = true;
  for (int k = 0; k < 2; ++k)
    vec = vec && aligned(p.src[k], 32) && (p.s_row[k] * e) % 32 == 0 && (p.s_head[k] * e) % 32 == 0;
  if (dtype == DFV_DTYPE_F32)
    return vec ? append_launch_t<float, true>(p, rows, stream)
               : append_launch_t<float, false>(p, rows, stream);
  return vec ? append_launch_t<__nv_bfloat16, true>(p, rows, stream)
             : append_launch_t<__nv_bfloat16, false>(p, rows, stream);
}

// ---------------------------------------------------------------- read back

struct Kv8ReadParams {
  dfv_kv8_cache c;
  int nblk;
  int pos0, end;
  void* dst[2];
  int64_t s_row, s_head;
  uint32_t* status;
};

template <typename T, int kN, bool kVec>
__device__ __forceinline__ void store_values(T* dst, const float* x) {
  if constexpr (!kVec) {
#pragma unroll
    for (int k = 0; k < kN; ++k) {
      if constexpr (sizeof(T) == 4) dst[k] = x[k];
      else dst[k] = __float2bfloat16_rn(x[k]);
    }
  } else if constexpr (sizeof(T) == 4) {
    if constexpr (kN == 16) {
      uint32_t w[16];
#pragma unroll
      for (int k = 0; k < 16; ++k) w[k] = __float_as_uint(x[k]);
      st32b(dst, w);
      st32b(dst + 8, w + 8);
    } else {
      *reinterpret_cast<float4*>(dst) = make_float4(x[0], x[1], x[2], x[3]);
    }
  } else if constexpr (kN == 16) {
    uint32_t w[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) w[k] = bf16x2_bits(x[2 * k], x[2 * k + 1]);
    st32b(dst, w);
  } else {
    *reinterpret_cast<uint2*>(dst) = make_uint2(bf16x2_bits(x[0], x[1]), bf16x2_bits(x[2], x[3]));
  }
}

// Code i of a row of codes, of which every byte has been flipped by 0x80:
// 0x4B0000uu is 2^23 + u.
__device__ __forceinline__ float code_at(const uint32_t* flipped, int i) {
  return __uint_as_float(__byte_perm(flipped[i >> 2], 0x4B000000u, 0x7440 | (i & 3))) - 8388736.0f;
}

template <typename T, int D, bool kVec>
__global__ void __launch_bounds__(D) kv8_read_kernel(const __grid_constant__ Kv8ReadParams p) {
  constexpr int kTpt = D / 64, kVt = D / 4;
  grid_dep_wait();
  grid_dep_launch_dependents();   // (after the wait: see common.cuh)
  const int C = p.c.state[0], held = p.c.state[2];
  const int tid = threadIdx.x, h = blockIdx.y, kv = blockIdx.z;
  // Rows behind the committed ones stay as they are, and rows of an open block
  // where the tail has others.
  int rows = C < 0 || C > p.c.capacity ? 0 : C;
  if (C / kBlk < held) rows = rows / kBlk * kBlk;
  const int end = min(p.end, rows);
  if (end < p.end && tid == 0 && blockIdx.x == 0 && h == 0 && kv == 0)
    report(p.status, DFV_DEV_CTX);
  const int b = p.pos0 / kBlk + blockIdx.x;
  const int first = max(p.pos0, b * kBlk), last = min(end, (b + 1) * kBlk);
  if (first >= last) return;
  T* dst = static_cast<T*>(p.dst[kv]) + h * p.s_head;
  if (b == C / kBlk) {   // the open block: bf16 rows
    const __nv_bfloat16* tail = static_cast<const __nv_bfloat16*>(kv ? p.c.v_tail : p.c.k_tail) +
                                (static_cast<int64_t>(h) * 2 + (b & 1)) * kBlk * D;
    // eight values a step and thread, all loads before the first store
    constexpr int kPer = D / 8;
    uint4 v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int row = (tid + k * D) / kPer;
      v[k] = *reinterpret_cast<const uint4*>(tail + row * D + (tid + k * D) % kPer * 8);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int pos = b * kBlk + (tid + k * D) / kPer;
      if (pos < first || pos >= last) continue;
      const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
      float x[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[2 * e] = bf16_lo(w[e]);
        x[2 * e + 1] = bf16_hi(w[e]);
      }
      T* o = dst + (pos - p.pos0) * p.s_row + (tid + k * D) % kPer * 8;
      store_values<T, 4, kVec>(o, x);
      store_values<T, 4, kVec>(o + 4, x + 4);
    }
    return;
  }
  const float scale = (kv ? p.c.v_scale : p.c.k_scale)[static_cast<int64_t>(h) * p.nblk + b];
  const int8_t* codes =
      (kv ? p.c.v_codes : p.c.k_codes) + static_cast<int64_t>(h) * p.nblk * kBlk * D;
  uint32_t q[16];
  if (kv == 0) {
    const int pos = b * kBlk + tid / kTpt;
    if (pos < first || pos >= last) return;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      *reinterpret_cast<uint4*>(q + 4 * j) = *reinterpret_cast<const uint4*>(
          codes + kv8_k_piece(b, tid / kTpt, tid % kTpt + j * kTpt, D));
#pragma unroll
    for (int j = 0; j < 16; ++j) q[j] ^= 0x80808080u;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float x[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = code_at(q + 4 * j, i) * scale;
      store_values<T, 16, kVec>(dst + (pos - p.pos0) * p.s_row + (tid % kTpt + j * kTpt) * 16, x);
    }
  } else {
    const int8_t* at = codes + kv8_v_piece(b, tid / kVt, tid % kVt * 4, D);
    ld32b(at, q);
    ld32b(at + 32, q + 8);
#pragma unroll
    for (int j = 0; j < 16; ++j) q[j] ^= 0x80808080u;
    const int pos0 = b * kBlk + tid / kVt * 16;
    T* o = dst + (pos0 - p.pos0) * p.s_row + tid % kVt * 4;
    const bool whole = pos0 >= first && pos0 + 16 <= last;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float x[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = code_at(q + 4 * j, i) * scale;
      if (whole || (pos0 + i >= first && pos0 + i < last))
        store_values<T, 4, kVec>(o + i * p.s_row, x);
    }
  }
}

template <typename T, bool kVec>
dfv_status read_launch_t(const Kv8ReadParams& p, cudaStream_t stream) {
  const dim3 grid((p.end - 1) / kBlk - p.pos0 / kBlk + 1, p.c.n_kv_heads, 2);
  switch (p.c.head_dim) {
    case 64: return launch_after(kv8_read_kernel<T, 64, kVec>, grid, 64, p, stream);
    case 128: return launch_after(kv8_read_kernel<T, 128, kVec>, grid, 128, p, stream);
    default: return launch_after(kv8_read_kernel<T, 256, kVec>, grid, 256, p, stream);
  }
}

}  // namespace dfv

extern "C" dfv_status dfv_kv8_append(const dfv_kv8_cache* cache, int at, int n_rows,
                                     const void* k_src, const void* v_src, int src_dtype,
                                     int64_t k_stride_row, int64_t k_stride_head,
                                     int64_t v_stride_row, int64_t v_stride_head,
                                     uint32_t* status, dfv_stream_t stream) {
  using namespace dfv;
  if (!kv8_cache_ok(cache)) return DFV_ERR_INVALID;
  if (!kv8_dim_ok(cache->head_dim)) return DFV_ERR_UNSUPPORTED;
  if (src_dtype != DFV_DTYPE_F32 && src_dtype != DFV_DTYPE_BF16) return DFV_ERR_UNSUPPORTED;
  const size_t size = src_dtype == DFV_DTYPE_F32 ? 4 : 2;
  if (at < -1 || n_rows < 0 || n_rows > cache->capacity ||
      static_cast<int64_t>(at < 0 ? 0 : at) + n_rows > cache->capacity)
    return DFV_ERR_INVALID;
  if (n_rows > 0 && (!k_src || !v_src || !aligned(k_src, size) || !aligned(v_src, size)))
    return DFV_ERR_INVALID;
  if (n_rows == 0 && at < 0) return DFV_OK;
  Kv8AppendParams p = {};
  p.c = *cache;
  p.at = at;
  p.n = n_rows;
  p.src[0] = k_src;
  p.src[1] = v_src;
  p.s_row[0] = k_stride_row;
  p.s_head[0] = k_stride_head;
  p.s_row[1] = v_stride_row;
  p.s_head[1] = v_stride_head;
  p.status = status;
  return kv8_append_launch(p, n_rows, src_dtype, static_cast<cudaStream_t>(stream));
}

extern "C" dfv_status dfv_kv8_commit(const dfv_kv8_cache* cache, int n_nodes,
                                     const int32_t* accept_len, const int32_t* path,
                                     const void* tree_k, const void* tree_v, uint32_t* status,
                                     dfv_stream_t stream) {
  using namespace dfv;
  if (!kv8_cache_ok(cache)) return DFV_ERR_INVALID;
  if (!kv8_dim_ok(cache->head_dim)) return DFV_ERR_UNSUPPORTED;
  if (n_nodes < 1 || n_nodes > kMaxNodes || !accept_len || !path || !tree_k || !tree_v ||
      !aligned(tree_k, 16) || !aligned(tree_v, 16))
    return DFV_ERR_INVALID;
  Kv8AppendParams p = {};
  p.c = *cache;
  p.at = -1;
  for (int k = 0; k < 2; ++k) {
    p.s_row[k] = static_cast<int64_t>(cache->n_kv_heads) * cache->head_dim;
    p.s_head[k] = cache->head_dim;
  }
  p.src[0] = tree_k;
  p.src[1] = tree_v;
  p.path = path;
  p.accept_len = accept_len;
  p.n_nodes = n_nodes;
  p.status = status;
  return kv8_append_launch(p, n_nodes, DFV_DTYPE_BF16, static_cast<cudaStream_t>(stream));
}

extern "C" dfv_status dfv_kv8_read(const dfv_kv8_cache* cache, int pos0, int n_rows, void* k_dst,
                                   void* v_dst, int dst_dtype, int64_t stride_row,
                                   int64_t stride_head, uint32_t* status, dfv_stream_t stream) {
  using namespace dfv;
  if (!kv8_cache_ok(cache)) return DFV_ERR_INVALID;
  if (!kv8_dim_ok(cache->head_dim)) return DFV_ERR_UNSUPPORTED;
  if (dst_dtype != DFV_DTYPE_F32 && dst_dtype != DFV_DTYPE_BF16) return DFV_ERR_UNSUPPORTED;
  if (pos0 < 0 || n_rows < 0 || static_cast<int64_t>(pos0) + n_rows > cache->capacity)
    return DFV_ERR_INVALID;
  if (n_rows == 0) return DFV_OK;
  const int e = dst_dtype == DFV_DTYPE_F32 ? 4 : 2;
  if (!k_dst || !v_dst || !aligned(k_dst, e) || !aligned(v_dst, e)) return DFV_ERR_INVALID;
  Kv8ReadParams p = {};
  p.c = *cache;
  p.nblk = kv8_blocks(cache->capacity);
  p.pos0 = pos0;
  p.end = pos0 + n_rows;
  p.dst[0] = k_dst;
  p.dst[1] = v_dst;
  p.s_row = stride_row;
  p.s_head = stride_head;
  p.status = status;
  const bool vec = aligned(k_dst, 32) && aligned(v_dst, 32) && (stride_row * e) % 32 == 0 &&
                   (stride_head * e) % 32 == 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dst_dtype == DFV_DTYPE_F32)
    return vec ? read_launch_t<float, true>(p, s) : read_launch_t<float, false>(p, s);
  return vec ? read_launch_t<__nv_bfloat16, true>(p, s) : read_launch_t<__nv_bfloat16, false>(p, s);
}
