// Eviction from a Q4_0 or F16 cache by the weight its keys have received, and
// rows of such a cache read back as values.
//
// Each KV head keeps, of its C rows, the first `sinks`, the last `recent`, and
// of the others the ones with the largest weight (ties to the lowest position);
// the rows keep their order and move bit for bit to another cache.
//
// The selection is an exact radix select: histograms of 11, 8, 8 and 5 bits of
// the weights' ordered bits find the smallest kept weight and how many equal ones
// are kept (it ends early where a whole bin stays; with 11 bits in the second one
// most of 2048 bins went to all CTAs, 4 us more for 131072 positions); a last pass
// counts in position order and writes the list. Pinned positions have the largest
// order of all.
// A head belongs to a cluster of up to 16 CTAs, each with its own run of
// positions, held in shared memory up to 16384 of them; they add their histograms
// up in each other's shared memory, so nothing goes through memory and no counter
// has to be reset. It is bound by latency: up to five rounds of about 2 us (4 heads
// of 131072 positions: 15 us; of 4097: 8). The copy is a gather of whole rows and
// bound by memory, as is reading back (32768 rows of 4 heads of 256: 17 and 33 us).

#include <atomic>

#include "common.cuh"

namespace dfv {

constexpr int kEvThreads = 1024;
constexpr int kEvWarps = kEvThreads / 32;
constexpr int kEvBins = 2048, kEvMore = 256;   // of the first pass, of a later one

struct EvictParams {
  int capacity, keep, sinks, recent, dst_capacity;
  const int32_t *ctx_len, *dropped;
  const float* weights;      // [head][capacity]
  int32_t* kept;             // [head][keep]
  float* weights_out;        // [head][dst_capacity], may be null
  int32_t *dst_ctx_len, *dst_dropped;
  uint32_t* status;
};

// Larger for larger weights; -0 equals +0, a NaN is below everything. The
// order of a number is in [0x7FFFFF, 0xFF800000], from which it comes back.
constexpr uint32_t kEvNan = 1, kEvPinned = 0xFFFFFFFFu, kEvNone = 0;
__device__ __forceinline__ uint32_t ev_order(float w) {
  const uint32_t u = __float_as_uint(w + 0.0f);
  const uint32_t o = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
  return w == w ? o : kEvNan;
}
__device__ __forceinline__ float ev_value(uint32_t o) {
  return __uint_as_float((o & 0x80000000u) ? (o & 0x7FFFFFFFu) : ~o);
}

__device__ __forceinline__ int ev_ctx(const EvictParams& p, bool tell) {
  const int C = *p.ctx_len;
  if (C >= 0 && C <= p.capacity) return C;
  if (tell) report(p.status, DFV_DEV_CTX);
  return max(0, min(C, p.capacity));
}

__device__ __forceinline__ void ev_remote_add(uint32_t* p, uint32_t v, int rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("red.relaxed.cluster.shared::cluster.add.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}
__device__ __forceinline__ void ev_cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

// A thread's orders stay in shared memory where its run is that short.
constexpr int kEvHeld = 16;
constexpr int kEvHeldBytes = kEvHeld * kEvThreads * 4;

template <bool kHeld>
__global__ void __launch_bounds__(kEvThreads, 1)
    evict_select_kernel(const __grid_constant__ EvictParams p) {
  __shared__ uint32_t s_hist[kEvBins];        // this CTA's
  __shared__ __align__(8) uint32_t s_all[kEvBins + 3 * kEvMore];   // the cluster's, by pass
  __shared__ uint32_t s_warp[2][kEvWarps], s_before[2];
  __shared__ uint32_t s_bin, s_above, s_inside;
  int cs, rank;
  asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(cs));
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  const int h = blockIdx.x / cs, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int b = tid; b < kEvBins + 3 * kEvMore; b += kEvThreads) s_all[b] = 0;
  if (tid < 2) s_before[tid] = 0;
  ev_cluster_sync();   // everyone's sums are zero
  grid_dep_wait();
  grid_dep_launch_dependents();   // (after the wait: see common.cuh)
  const int C = ev_ctx(p, blockIdx.x == 0 && tid == 0);
  const int n = min(C, p.keep);
  if (blockIdx.x == 0 && tid == 0) {
    *p.dst_ctx_len = n;
    if (p.dst_dropped) *p.dst_dropped = (p.dropped ? *p.dropped : 0) + (C - n);
  }
  const float* w = p.weights + static_cast<int64_t>(h) * p.capacity;
  int32_t* kept = p.kept + static_cast<int64_t>(h) * p.keep;
  // Pinned positions count as the largest of all: together they are at most
  // `need`, so that a position's place depends on its order alone.
  const bool all = C <= p.keep;
  const int s0 = p.sinks, s1 = C - p.recent;
  uint32_t need = all ? 0 : static_cast<uint32_t>(p.keep);
  // each CTA has a run of positions, each of its warps a run of that
  const int lo = static_cast<int>(static_cast<int64_t>(C) * rank / cs);
  const int hi = static_cast<int>(static_cast<int64_t>(C) * (rank + 1) / cs);
  const int steps = ((hi - lo + kEvWarps - 1) / kEvWarps + 31) / 32;
  const int j0 = min(hi, lo + warp * steps * 32), j1 = min(hi, j0 + steps * 32);
  auto order = [&](int i) {
    const int j = j0 + i * 32 + lane;
    const uint32_t o = ev_order(w[min(j, C - 1)]);   // (no branch: loads in a row)
    return j >= j1 ? kEvNone : j < s0 || j >= s1 ? kEvPinned : o;
  };
  extern __shared__ uint32_t s_held[];   // [step][thread]
  if constexpr (kHeld) {
#pragma unroll 8
    for (int i = 0; i < steps; ++i) s_held[i * kEvThreads + tid] = order(i);
  }
  auto each = [&](auto f) {   // f(step, order): every lane of the warp
#pragma unroll 4
    for (int i = 0; i < steps; ++i) {
      if constexpr (kHeld) f(i, s_held[i * kEvThreads + tid]);
      else f(i, order(i));
    }
  };
  // Sum over the warps before this one, and over all; s_warp[k] holds each warp's.
  auto warps_before = [&](int k, uint32_t& total) {
    uint32_t v = s_warp[k][lane];
    const uint32_t mine = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t u = __shfl_up_sync(0xFFFFFFFFu, v, o);
      if (lane >= o) v += u;
    }
    total = __shfl_sync(0xFFFFFFFFu, v, 31);
    return __shfl_sync(0xFFFFFFFFu, v - mine, warp);
  };

  // ---- the smallest kept order, 11, 8, 8 and 5 bits at a time
  uint32_t prefix = 0;   // (all: every order is above it)
  if (need > 0) {
    int known = 0;   // leading bits of `prefix` that are found
#pragma unroll 1
    for (int pass = 0; known < 32; ++pass) {
      const int bits = pass == 0 ? 11 : pass < 3 ? 8 : 5, shift = 32 - known - bits;
      const int bins = 1 << bits;
      uint32_t* sums = s_all + (pass == 0 ? 0 : kEvBins + (pass - 1) * kEvMore);
      for (int b = tid; b < bins; b += kEvThreads) s_hist[b] = 0;
      __syncthreads();
      const uint32_t mask = pass == 0 ? 0 : 0xFFFFFFFFu << (32 - known);
      each([&](int, uint32_t o) {   // (kEvNone is in a lower bin than any, or below in the same)
        if ((o & mask) == prefix) atomicAdd(&s_hist[(o >> shift) & (bins - 1)], 1u);
      });
      __syncthreads();
      // few of the first pass's bins are not empty: they are added up in every CTA
      for (int b = tid; b < bins; b += kEvThreads) {
        const uint32_t v = s_hist[b];
        if (v)
          for (int r = 0; r < cs; ++r) ev_remote_add(&sums[b], v, r);
      }
      ev_cluster_sync();
      // bins from the largest down, two a thread: where the count reaches `need`
      uint2 two = make_uint2(0, 0);
      if (2 * tid < bins) two = *reinterpret_cast<const uint2*>(&sums[bins - 2 - 2 * tid]);
      const uint32_t c[2] = {two.y, two.x};
      uint32_t sum = c[0] + c[1];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, sum, o);
        if (lane >= o) sum += v;
      }
      if (lane == 31) s_warp[0][warp] = sum;
      __syncthreads();
      uint32_t total;
      uint32_t above = warps_before(0, total) + sum - c[0] - c[1];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        if (above < need && need <= above + c[k]) {   // one thread's
          s_bin = bins - 1 - (2 * tid + k);
          s_above = above;
          s_inside = c[k];
        }
        above += c[k];
      }
      __syncthreads();
      need -= s_above;
      prefix |= s_bin << shift;
      known += bits;
      if (need == s_inside && prefix > 0) {   // the whole bin stays: all above what is below it
        prefix -= 1;
        need = 0;
        break;
      }
    }
  }
  // What is above `prefix` stays, and the first `need` of what equals it.

  // ---- the list, in position order
  uint32_t n_over = 0, n_same = 0;
  each([&](int, uint32_t o) {
    n_over += o > prefix ? 1 : 0;
    n_same += o == prefix ? 1 : 0;
  });
  n_over = __reduce_add_sync(0xFFFFFFFFu, n_over);
  n_same = __reduce_add_sync(0xFFFFFFFFu, n_same);
  __syncthreads();   // s_warp has been read
  if (lane == 0) {
    s_warp[0][warp] = n_over;
    s_warp[1][warp] = n_same;
  }
  __syncthreads();
  uint32_t t_over, t_same;
  uint32_t at_over = warps_before(0, t_over), at_same = warps_before(1, t_same);
  // a CTA adds its counts for those behind it
  if (tid > rank && tid < cs) {
    ev_remote_add(&s_before[0], t_over, tid);
    ev_remote_add(&s_before[1], t_same, tid);
  }
  ev_cluster_sync();
  at_over += s_before[0];
  at_same += s_before[1];
  float* out = p.weights_out ? p.weights_out + static_cast<int64_t>(h) * p.dst_capacity : nullptr;
  each([&](int i, uint32_t o) {
    const bool over = o > prefix, same = o == prefix;
    const unsigned bo = __ballot_sync(0xFFFFFFFFu, over), bs = __ballot_sync(0xFFFFFFFFu, same);
    const unsigned below = (1u << lane) - 1u;
    uint32_t es = at_same;
    if (bs) {   // hardly ever
      es += __popc(bs & below);
      at_same += __popc(bs);
    }
    if (over || (same && es < need)) {
      const uint32_t at = at_over + __popc(bo & below) + min(es, need);
      const int j = j0 + i * 32 + lane;
      kept[at] = j;
      if (out) out[at] = o == kEvPinned || o == kEvNan ? w[j] : ev_value(o);
    }
    at_over += __popc(bo);
  });
}

struct MoveParams {
  int heads, capacity, dst_capacity, keep;
  const int32_t* ctx_len;
  const int32_t* kept;
  const uint8_t *k, *v;
  uint8_t *k_out, *v_out;
};

// One piece (4, 8 or 16 bytes) of a kept row per thread and step: writes are
// contiguous, reads whole rows. kPieces is known for Q4_0 (9 pieces of D / 16
// bytes), a power of two else.
template <typename V, int kPieces>
__global__ void __launch_bounds__(256) evict_move_kernel(const __grid_constant__ MoveParams p) {
  grid_dep_wait();
  grid_dep_launch_dependents();   // (after the wait: see common.cuh)
  const int C = max(0, min(*p.ctx_len, p.capacity));
  const int n = min(C, p.keep);
  const int64_t per_head = static_cast<int64_t>(n) * kPieces;
  const int h = blockIdx.y;
  const uint8_t* src = (blockIdx.z ? p.v : p.k);
  uint8_t* dst = (blockIdx.z ? p.v_out : p.k_out);
  const V* s = reinterpret_cast<const V*>(src) + static_cast<int64_t>(h) * p.capacity * kPieces;
  V* d = reinterpret_cast<V*>(dst) + static_cast<int64_t>(h) * p.dst_capacity * kPieces;
  const int32_t* kept = p.kept + static_cast<int64_t>(h) * p.keep;
  constexpr int kAhead = 4;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * 256;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < per_head;
       i += kAhead * stride) {
    V x[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int64_t k = i + u * stride;
      if (k >= per_head) break;
      const int64_t row = k / kPieces;
      x[u] = s[static_cast<int64_t>(kept[row]) * kPieces + (k - row * kPieces)];
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int64_t k = i + u * stride;
      if (k < per_head) d[k] = x[u];
    }
  }
}

struct ReadRowsParams {
  int heads, head_dim, capacity, pos0, n_rows;
  const uint8_t *k, *v;
  void *k_dst, *v_dst;
  int64_t stride_row, stride_head;
};

template <bool kVec>
__device__ __forceinline__ void put8(float* d, const float* x) {
  if constexpr (kVec) {
    reinterpret_cast<float4*>(d)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(d)[1] = make_float4(x[4], x[5], x[6], x[7]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) d[i] = x[i];
  }
}
template <bool kVec>
__device__ __forceinline__ void put8(__nv_bfloat16* d, const float* x) {
  if constexpr (kVec) {
    uint4 o;
    uint32_t* w = reinterpret_cast<uint32_t*>(&o);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    *reinterpret_cast<uint4*>(d) = o;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) d[i] = __float2bfloat16_rn(x[i]);
  }
}

// Eight values of a row per thread, several rows in flight; a row's threads are
// neighbours, so writes are contiguous (kVec: 16 bytes each).
template <typename T, bool kF16, bool kVec>
__global__ void __launch_bounds__(256) read_rows_kernel(const __grid_constant__ ReadRowsParams p) {
  constexpr int kAhead = 4;
  grid_dep_wait();
  grid_dep_launch_dependents();   // (after the wait: see common.cuh)
  const int shift = p.head_dim == 256 ? 5 : p.head_dim == 128 ? 4 : 3;   // threads of a row
  const int g = threadIdx.x & ((1 << shift) - 1), h = blockIdx.y;
  const int rows = 256 >> shift, step = gridDim.x * rows;
  const int64_t row_bytes = kv_row_bytes(kF16 ? DFV_KV_F16 : DFV_KV_Q4_0, p.head_dim);
  const uint8_t* src = (blockIdx.z ? p.v : p.k) +
                       (static_cast<int64_t>(h) * p.capacity + p.pos0) * row_bytes;
  T* dst = static_cast<T*>(blockIdx.z ? p.v_dst : p.k_dst) + h * p.stride_head + g * 8;
  // dims [8 g, + 8) of a Q4_0 block: low nibbles of its first 16 values, high of its last
  const int off = kF16 ? g * 16 : (g >> 2) * 18, nib = (g & 2) ? 4 : 0, word = 1 + (g & 1) * 4;
  for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * rows + (threadIdx.x >> shift);
       r0 < p.n_rows; r0 += static_cast<int64_t>(kAhead) * step) {
    uint32_t in[kAhead][5];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int64_t r = r0 + static_cast<int64_t>(u) * step;
      if (r >= p.n_rows) break;
      const uint8_t* a = src + r * row_bytes + off;
      if constexpr (kF16) {
        const uint4 v = *reinterpret_cast<const uint4*>(a);
        in[u][0] = v.x, in[u][1] = v.y, in[u][2] = v.z, in[u][3] = v.w;
      } else {
        const uint16_t* b = reinterpret_cast<const uint16_t*>(a);
        in[u][4] = b[0];
#pragma unroll
        for (int e = 0; e < 4; ++e) in[u][e] = b[word + e];
      }
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int64_t r = r0 + static_cast<int64_t>(u) * step;
      if (r >= p.n_rows) break;
      float x[8];
      if constexpr (kF16) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&in[u][e]));
          x[2 * e] = f.x;
          x[2 * e + 1] = f.y;
        }
      } else {
        const float d = __half2float(__ushort_as_half(static_cast<uint16_t>(in[u][4])));
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t c = in[u][e] >> nib;
          x[2 * e] = (static_cast<float>(c & 15u) - 8.0f) * d;
          x[2 * e + 1] = (static_cast<float>((c >> 8) & 15u) - 8.0f) * d;
        }
      }
      put8<kVec>(dst + r * p.stride_row, x);
    }
  }
}

template <typename F, typename P>
dfv_status launch_after(F* kernel, const P& p, dim3 grid, int threads, cudaStream_t stream,
                        int cluster = 1, int smem = 0) {
  cudaLaunchConfig_t cfg = {};
  cfg.dynamicSmemBytes = smem;
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, p) == cudaSuccess ? DFV_OK : DFV_ERR_CUDA;
}

template <typename V, int kPieces>
dfv_status move_launch(const MoveParams& p, cudaStream_t stream) {
  // about eight CTAs an SM over heads, K and V; four pieces a thread at a time
  const int64_t want = (static_cast<int64_t>(p.keep) * kPieces + 1023) / 1024;
  const int64_t most = (static_cast<int64_t>(sm_count()) * 8 + 2 * p.heads - 1) / (2 * p.heads);
  const int64_t x = want < most ? want : most;
  return launch_after(evict_move_kernel<V, kPieces>, p,
                      dim3(static_cast<unsigned>(x < 1 ? 1 : x), p.heads, 2), 256, stream);
}

template <typename T, bool kF16>
dfv_status read_launch(const ReadRowsParams& p, dim3 grid, bool vec, cudaStream_t stream) {
  return vec ? launch_after(read_rows_kernel<T, kF16, true>, p, grid, 256, stream)
             : launch_after(read_rows_kernel<T, kF16, false>, p, grid, 256, stream);
}

}  // namespace dfv

extern "C" dfv_status dfv_kv_evict(int n_kv_heads, int head_dim, int kv_format,
                                   int cache_capacity, const int32_t* ctx_len,
                                   const int32_t* dropped, const void* k_cache,
                                   const void* v_cache, const float* weights, int keep, int sinks,
                                   int recent, int dst_capacity, void* k_dst, void* v_dst,
                                   int32_t* dst_ctx_len, int32_t* dst_dropped,
                                   float* weights_out, int32_t* kept, uint32_t* status,
                                   dfv_stream_t stream) {
  using namespace dfv;
  if ((kv_format != DFV_KV_Q4_0 && kv_format != DFV_KV_F16) ||
      (head_dim != 64 && head_dim != 128 && head_dim != 256))
    return DFV_ERR_UNSUPPORTED;
  if (n_kv_heads < 1 || n_kv_heads > 65535 || cache_capacity < 1 ||
      cache_capacity > (1 << 30) || keep < 1 || keep > dst_capacity || sinks < 0 || recent < 0 ||
      static_cast<int64_t>(sinks) + recent > keep || dst_capacity > (1 << 30))
    return DFV_ERR_INVALID;
  if (!ctx_len || !k_cache || !v_cache || !weights || !k_dst || !v_dst || !dst_ctx_len || !kept ||
      !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(k_dst, 16) ||
      !aligned(v_dst, 16) || !aligned(weights, 4) || !aligned(weights_out, 4) ||
      !aligned(kept, 4) || !aligned(ctx_len, 4) || !aligned(dst_ctx_len, 4) ||
      !aligned(dropped, 4) || !aligned(dst_dropped, 4))
    return DFV_ERR_INVALID;
  if (k_dst == k_cache || v_dst == v_cache || k_dst == v_cache || v_dst == k_cache ||
      k_dst == v_dst || dst_ctx_len == ctx_len || weights_out == weights)
    return DFV_ERR_INVALID;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const EvictParams e = {cache_capacity, keep, sinks, recent, dst_capacity, ctx_len, dropped,
                         weights, kept, weights_out, dst_ctx_len, dst_dropped, status};
  // A CTA for about 2048 positions of a head, eight at most; for few heads
  // sixteen (such a cluster lies in one GPC, so only some run at a time: select
  // and copy of one head of 131072 positions 15.2 us, by eight 18.1; of eight
  // heads 28.5 and 20.2).
  const int most = n_kv_heads <= 4 ? 16 : 8;
  int cs = 1;
  while (cs < most && cache_capacity > cs * 2048) cs <<= 1;
  static std::atomic<int> configured[64];   // per device
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return DFV_ERR_CUDA;
  if (!configured[dev].load(std::memory_order_acquire)) {
    if (cudaFuncSetAttribute(evict_select_kernel<true>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kEvHeldBytes) != cudaSuccess ||
        cudaFuncSetAttribute(evict_select_kernel<true>,
                             cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess ||
        cudaFuncSetAttribute(evict_select_kernel<false>,
                             cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
      return DFV_ERR_CUDA;
    configured[dev].store(1, std::memory_order_release);
  }
  // (a warp's run is rounded up to whole steps of 32)
  const int run = (cache_capacity - 1) / cs + 1;
  const int steps = ((run - 1) / kEvWarps + 32) / 32;
  const dim3 grid(n_kv_heads * cs);
  const dfv_status st =
      steps <= kEvHeld ? launch_after(evict_select_kernel<true>, e, grid, kEvThreads, s, cs,
                                      steps * kEvThreads * 4)
                       : launch_after(evict_select_kernel<false>, e, grid, kEvThreads, s, cs);
  if (st != DFV_OK) return st;
  const MoveParams m = {n_kv_heads, cache_capacity, dst_capacity, keep, ctx_len, kept,
                        static_cast<const uint8_t*>(k_cache), static_cast<const uint8_t*>(v_cache),
                        static_cast<uint8_t*>(k_dst), static_cast<uint8_t*>(v_dst)};
  if (kv_format == DFV_KV_F16)
    return head_dim == 64    ? move_launch<uint4, 8>(m, s)
           : head_dim == 128 ? move_launch<uint4, 16>(m, s)
                             : move_launch<uint4, 32>(m, s);
  return head_dim == 64    ? move_launch<uint32_t, 9>(m, s)
         : head_dim == 128 ? move_launch<uint2, 9>(m, s)
                           : move_launch<uint4, 9>(m, s);
}

extern "C" dfv_status dfv_kv_read_rows(int n_kv_heads, int head_dim, int kv_format,
                                       int cache_capacity, int pos0, int n_rows,
                                       const void* k_cache, const void* v_cache, void* k_dst,
                                       void* v_dst, int dst_dtype, int64_t stride_row,
                                       int64_t stride_head, dfv_stream_t stream) {
  using namespace dfv;
  if ((kv_format != DFV_KV_Q4_0 && kv_format != DFV_KV_F16) ||
      (head_dim != 64 && head_dim != 128 && head_dim != 256) ||
      (dst_dtype != DFV_DTYPE_F32 && dst_dtype != DFV_DTYPE_BF16))
    return DFV_ERR_UNSUPPORTED;
  if (n_kv_heads < 1 || n_kv_heads > 65535 || cache_capacity < 1 || pos0 < 0 || n_rows < 0 ||
      static_cast<int64_t>(pos0) + n_rows > cache_capacity)
    return DFV_ERR_INVALID;
  if (n_rows == 0) return DFV_OK;
  const size_t size = dst_dtype == DFV_DTYPE_F32 ? 4 : 2;
  if (!k_cache || !v_cache || !k_dst || !v_dst || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
      !aligned(k_dst, size) || !aligned(v_dst, size))
    return DFV_ERR_INVALID;
  const ReadRowsParams p = {n_kv_heads, head_dim, cache_capacity, pos0, n_rows,
                            static_cast<const uint8_t*>(k_cache),
                            static_cast<const uint8_t*>(v_cache), k_dst, v_dst, stride_row,
                            stride_head};
  const int64_t want = (static_cast<int64_t>(n_rows) * (head_dim / 8) + 1023) / 1024;
  const int64_t most = (static_cast<int64_t>(sm_count()) * 8 + 2 * n_kv_heads - 1) /
                       (2 * n_kv_heads);
  const dim3 grid(static_cast<unsigned>(want < most ? want : most), n_kv_heads, 2);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int64_t e16 = static_cast<int64_t>(16 / size);
  const bool vec = aligned(k_dst, 16) && aligned(v_dst, 16) && stride_row % e16 == 0 &&
                   stride_head % e16 == 0;
  if (kv_format == DFV_KV_F16)
    return dst_dtype == DFV_DTYPE_F32 ? read_launch<float, true>(p, grid, vec, s)
                                      : read_launch<__nv_bfloat16, true>(p, grid, vec, s);
  return dst_dtype == DFV_DTYPE_F32 ? read_launch<float, false>(p, grid, vec, s)
                                    : read_launch<__nv_bfloat16, false>(p, grid, vec, s);
}
