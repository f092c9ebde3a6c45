// Log probabilities of given tokens, the entropy of each row of logits and
// its top alternatives.
//
//   m = max_i x_i, z_i = x_i - m, s = sum exp(z_i)
//   log p(t) = z_t - log s
//   entropy  = log s - (sum exp(z_i) z_i) / s
//   top      = the `top` largest x, ties to the lowest index
//
// Everything comes from one pass over the row: each thread carries a running
// (m, s, sum exp(z) z), rescaled when its maximum moves, and the partial
// triples are merged in a fixed order. The kernel is bound by memory for many
// rows and by latency for few, so a row belongs to a cluster of 1 to 16 CTAs
// that write their results into the first one's shared memory (one launch, no
// workspace, nothing to reset). Few rows get CTAs of 1024 threads: a slice of
// 152 K logits then is one round of loads.
//
// The alternatives cost little beside that pass. The first chunk of
// a slice (its values stay in registers) is cut into 64 groups; the top-th
// largest of the group maxima is a lower bound of the slice's top-th value,
// and whatever reaches that bound is collected in shared memory. The bound is
// renewed from the candidates as the slice goes on, so that a row in random
// order collects a few times `top` of them per renewal. Rows that collect more
// than the buffer holds (many equal values, ascending values) are read once
// more by a path that cuts the buffer back to the best `top` as it fills.
// Candidates are ordered by a 64-bit key (value, then lower index), which is
// unique, so the result does not depend on the order of collection.

#include <atomic>
#include <climits>
#include <cooperative_groups.h>

#include "common.cuh"

namespace dfv {

namespace cg = cooperative_groups;

constexpr int kLpGroups = 64;       // >= DFV_MAX_TOP
constexpr int kLpCap = 1024;        // candidates a CTA can hold
constexpr int kLpMaxCluster = 16;
constexpr int kLpVecs = 4;          // 16-byte loads per thread and chunk
constexpr float kLog2e = 1.4426950408889634f;

struct LogprobParams {
  int vocab, top;
  const void* logits;
  int64_t stride;
  const int32_t* tokens;
  float* logprob;
  float* entropy;
  int32_t* top_ids;
  float* top_logprobs;
  uint32_t* status;
};

__device__ __forceinline__ float lp_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Maxima that are NaN if an operand is: a thread that has seen nothing but -inf
// learns of a NaN only by them.
__device__ __forceinline__ float lp_max3(float a, float b, float c) {
  float y;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
__device__ __forceinline__ float lp_max(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}
// at least -200, and NaN if x is
__device__ __forceinline__ float lp_floor(float x) {
  float y;
  asm("max.NaN.f32 %0, %1, 0fC3480000;" : "=f"(y) : "f"(x));
  return y;
}

// Two float32 operations in one instruction.
__device__ __forceinline__ float2 lp_add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "add.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 lp_mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "mul.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 lp_fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, c;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "mov.b64 c, {%6, %7};\n\tfma.rn.f32x2 a, a, b, c;\n\tmov.b64 {%0, %1}, a;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}

// Orders like (value, lower index first); -0 equals +0.
__device__ __forceinline__ uint64_t lp_key(float x, int idx) {
  uint32_t u = __float_as_uint(x + 0.0f);
  u = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
  return (static_cast<uint64_t>(u) << 32) | static_cast<uint32_t>(~idx);
}
__device__ __forceinline__ float lp_value(uint64_t key) {
  const uint32_t u = static_cast<uint32_t>(key >> 32);
  return __uint_as_float((u & 0x80000000u) ? (u & 0x7FFFFFFFu) : ~u);
}
__device__ __forceinline__ int lp_index(uint64_t key) {
  return static_cast<int>(~static_cast<uint32_t>(key));
}

// Running maximum, sum of exp(x - m) and of exp(x - m) (x - m).
struct LpStats {
  float m, s, t;
  __device__ __forceinline__ void init() {
    m = -INFINITY;
    s = 0.0f;
    t = 0.0f;
  }
  __device__ __forceinline__ void raise(float to) {   // to > m
    const float d = fmaxf(m - to, -200.0f);           // exp(-200) is zero; 0 * -inf is not
    const float f = lp_ex2(d * kLog2e);
    t = f * fmaf(d, s, t);
    s *= f;
    m = to;
  }
  // All 32 lanes' triples joined, in every lane: one common maximum, then sums
  // by exchanges whose order is fixed.
  __device__ __forceinline__ void warp_join() {
    float to;
    asm volatile("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(to) : "f"(m));
    if (to > m) raise(to);
    else if (to != to) m = s = t = NAN;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
      t += __shfl_xor_sync(0xFFFFFFFFu, t, o);
    }
  }
};

template <typename T> struct LpVec;   // one 16-byte load
template <> struct LpVec<float> {
  static constexpr int kN = 4;
  static __device__ __forceinline__ float at(const uint4& v, int i) {
    return __uint_as_float(i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w);
  }
};
template <> struct LpVec<__nv_bfloat16> {
  static constexpr int kN = 8;
  static __device__ __forceinline__ float at(const uint4& v, int i) {
    const uint32_t w = i < 2 ? v.x : i < 4 ? v.y : i < 6 ? v.z : v.w;
    return __uint_as_float(i & 1 ? w & 0xFFFF0000u : w << 16);
  }
};

__device__ __forceinline__ float lp_to_f32(float x) { return x; }
__device__ __forceinline__ float lp_to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }

struct LpSmem {
  uint64_t buf[kLpCap];
  uint64_t gkey[kLpGroups];
  uint64_t best[DFV_MAX_TOP];   // the slice's, in order
  alignas(16) float gmax[kLpGroups];
  LpStats wst[32];
  LpStats st;
  uint64_t cut;
  float bound;
  int count, n_best;
  // the cluster's slices, written by their CTAs (first CTA only)
  LpStats cst[kLpMaxCluster];
  int cn[kLpMaxCluster];
  uint64_t cbest[kLpMaxCluster][DFV_MAX_TOP];
};

// Adds kN values with maximum vm (all of one thread) to its statistics.
template <int kN, typename F>
__device__ __forceinline__ void lp_add(LpStats& st, float vm, F value) {
  if (!(vm <= st.m)) {
    if (vm == vm) st.raise(vm);
    else st.m = st.s = st.t = NAN;   // NaN stays: comparisons with it fail
  }
  if (st.m == -INFINITY) return;     // nothing but -inf so far
  float2 s2 = make_float2(0.0f, 0.0f), t2 = s2;
  const float2 m2 = make_float2(-st.m, -st.m), c2 = make_float2(kLog2e, kLog2e);
#pragma unroll
  for (int i = 0; i < kN; i += 2) {
    float2 z = lp_add2(make_float2(value(i), kN > 1 ? value(i + 1) : -INFINITY), m2);
    // exp(-200) is zero; the limit keeps 0 * -inf out of the sum
    z.x = lp_floor(z.x);
    z.y = lp_floor(z.y);
    const float2 y = lp_mul2(z, c2);
    const float2 e = make_float2(lp_ex2(y.x), lp_ex2(y.y));
    s2 = lp_add2(s2, e);
    t2 = lp_fma2(e, z, t2);
  }
  st.s += s2.x + s2.y;
  st.t += t2.x + t2.y;
}

__device__ __forceinline__ void lp_push(LpSmem& sm, float x, int idx) {
  const int k = atomicAdd(&sm.count, 1);
  if (k < kLpCap) sm.buf[k] = lp_key(x, idx);
}

// The best `top` of buf[0, c), in order, into sm.best (n_best of them).
// All threads; c <= kLpCap. Large sets are cut first: at least `top` keys
// reach the top-th largest of the group maxima.
template <int kLpThreads>
__device__ void lp_select(LpSmem& sm, int c, int top) {
  const int tid = threadIdx.x;
  while (c > 128) {
    uint64_t mine = 0;
    for (int i = tid; i < c; i += kLpThreads) mine = max(mine, sm.buf[i]);
    uint64_t* all = sm.gkey;
    if (tid < kLpGroups) all[tid] = 0;
    __syncthreads();
    atomicMax(reinterpret_cast<unsigned long long*>(&all[tid % kLpGroups]),
              static_cast<unsigned long long>(mine));
    __syncthreads();
    if (tid < kLpGroups) {
      int above = 0;
      for (int i = 0; i < kLpGroups; ++i) above += all[i] > all[tid];
      if (above == top - 1) sm.cut = all[tid];
    }
    __syncthreads();
    const uint64_t cut = sm.cut;
    constexpr int kKeep = kLpCap / kLpThreads;
    uint64_t keep[kKeep];
    int n = 0;
#pragma unroll
    for (int j = 0; j < kKeep; ++j) {
      const int i = tid + j * kLpThreads;
      keep[j] = i < c ? sm.buf[i] : 0;
      n += keep[j] >= cut && keep[j] != 0;
    }
    if (tid == 0) sm.count = 0;
    __syncthreads();
    int at = n ? atomicAdd(&sm.count, n) : 0;
#pragma unroll
    for (int j = 0; j < kKeep; ++j)
      if (keep[j] >= cut && keep[j] != 0) sm.buf[at++] = keep[j];
    __syncthreads();
    const int left = sm.count;
    __syncthreads();
    if (left == c) break;
    c = left;
  }
  const int n_best = min(c, top);
  for (int i = tid; i < c; i += kLpThreads) {
    const uint64_t mine = sm.buf[i];
    int above = 0;
#pragma unroll 8
    for (int k = 0; k < c; ++k) above += sm.buf[k] > mine;
    if (above < top) sm.best[above] = mine;
  }
  if (tid == 0) sm.n_best = n_best;
  __syncthreads();
}

__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int kPending>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kPending) : "memory");
}

__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

template <typename T, int kLpThreads>
__global__ void __launch_bounds__(kLpThreads, 1024 / kLpThreads)
    logprob_kernel(const __grid_constant__ LogprobParams p) {
  __shared__ LpSmem sm;
  constexpr int kV = LpVec<T>::kN;
  cg::cluster_group cl = cg::this_cluster();
  const int cs = cl.num_blocks(), rank = cl.block_rank();
  const int row = blockIdx.x / cs, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const T* x = static_cast<const T*>(p.logits) + row * p.stride;
  // The row: a head before the first 16-byte boundary, whole vectors, a
  // tail. The vectors are dealt in equal runs; the first CTA of the cluster
  // has the head too, the last one the tail.
  const int over = static_cast<int>(reinterpret_cast<uintptr_t>(x) & 15);   // bytes past one
  const int head = min(p.vocab, (16 - over) % 16 / static_cast<int>(sizeof(T)));
  const int nv = (p.vocab - head) / kV;
  const int v0 = static_cast<int>(static_cast<int64_t>(nv) * rank / cs);
  const int v1 = static_cast<int>(static_cast<int64_t>(nv) * (rank + 1) / cs);
  const uint4* xv = reinterpret_cast<const uint4*>(x + head);
  int extra = -1;   // this thread's element outside the vectors
  if (rank == 0 && tid < head) extra = tid;
  if (rank == cs - 1 && tid >= 32 && tid - 32 < p.vocab - head - nv * kV)
    extra = head + nv * kV + tid - 32;
  const int slice_n = (v1 - v0) * kV + (rank == 0 ? head : 0) +
                      (rank == cs - 1 ? p.vocab - head - nv * kV : 0);
  const int top = p.top;
  if (tid == 0) {
    sm.count = 0;
    sm.bound = -INFINITY;   // stays where too many groups hold a NaN
  }
  if (cs > 1) cluster_arrive();   // waited for before the first CTA's memory is written
  grid_dep_wait();   // set up under the kernel before; nothing has been read yet
  grid_dep_launch_dependents();   // (after the wait: see common.cuh)

  // the given token and its logit, read meanwhile
  int token = 0;
  float x_token = NAN;
  if (tid == 0 && rank == 0 && p.logprob) {
    token = p.tokens[row];
    if (token >= 0 && token < p.vocab) x_token = lp_to_f32(x[token]);
    else report(p.status, DFV_DEV_BAD_TOKEN);
  }
  LpStats st;
  st.init();
  constexpr int kStep = kLpThreads * kLpVecs;
  constexpr bool kAhead = kLpThreads == 128 && sizeof(T) == 2;
  uint4 v[kLpVecs];
  const uint32_t lowest = sizeof(T) == 4 ? 0xFF800000u : 0xFF80FF80u;   // -inf
  const uint4 none = make_uint4(lowest, lowest, lowest, lowest);
  auto load = [&](int base) {
#pragma unroll
    for (int j = 0; j < kLpVecs; ++j) {
      const int i = base + j * kLpThreads + tid;
      v[j] = i < v1 ? xv[i] : none;
    }
  };
  // 16-bit rows in CTAs of 128 threads: whole chunks come by way of shared
  // memory, each thread copying its own vectors of the next chunk before it
  // works on this one, so that loads are in flight throughout (1024 x 151936,
  // top 5: 64 us, by loads to registers 70; f32 rows, which are bound by
  // memory already: 112 to 117 for 99). A slot is overwritten only after the
  // values read from it have been used.
  __shared__ uint4 ring[kAhead ? 2 * kStep : 1];
  auto fetch = [&](int base, int slot) {
    if (base + kStep <= v1) {
#pragma unroll
      for (int j = 0; j < kLpVecs; ++j)
        cp_async16(&ring[(slot * kLpVecs + j) * kLpThreads + tid],
                   xv + base + j * kLpThreads + tid);
    }
    cp_async_commit();
  };
  const uint4* mine = xv + tid;
  auto load_full = [&](int base) {
#pragma unroll
    for (int j = 0; j < kLpVecs; ++j) v[j] = mine[base + j * kLpThreads];
  };
  auto value = [&](int i) { return LpVec<T>::at(v[i / kV], i % kV); };
  float jm[kLpVecs];   // maximum of each vector
  auto chunk_max = [&]() {
#pragma unroll
    for (int j = 0; j < kLpVecs; ++j) {
      jm[j] = lp_max3(value(j * kV), value(j * kV + 1), value(j * kV + 2));
#pragma unroll
      for (int e = 3; e < kV; e += 2)
        jm[j] = lp_max3(jm[j], value(j * kV + e), value(j * kV + (e + 1 < kV ? e + 1 : e)));
    }
    static_assert(kLpVecs == 4, "maximum of four");
    return lp_max(lp_max3(jm[0], jm[1], jm[2]), jm[3]);
  };
  auto push_from = [&](int base, float bound) {
#pragma unroll
    for (int j = 0; j < kLpVecs; ++j) {
      if (!(jm[j] >= bound)) continue;
      const int i = base + j * kLpThreads + tid;
#pragma unroll
      for (int e = 0; e < kV; ++e) {
        const float w = LpVec<T>::at(v[j], e);
        if (w >= bound && i < v1) lp_push(sm, w, head + i * kV + e);
      }
    }
  };

  // The top-th largest of 4 * quads group maxima, which as many values reach.
  auto raise_bound = [&](float g, int quads) {
    const float4* all = reinterpret_cast<const float4*>(sm.gmax);
    int above = 0, same = 0;
#pragma unroll 4
    for (int k = 0; k < quads; ++k) {
      const float4 o = all[k];
      above += (o.x > g) + (o.y > g) + (o.z > g) + (o.w > g);
      same += (o.x >= g) + (o.y >= g) + (o.z >= g) + (o.w >= g);
    }
    if (above < top && same >= top) sm.bound = g;   // the same value from each such thread
  };

  // ---- first chunk: statistics, and the bound for the alternatives
  load(v0);
  if constexpr (kAhead) fetch(v0 + kStep, 0);
  const float xe = extra >= 0 ? lp_to_f32(x[extra]) : -INFINITY;
  float vm = chunk_max();
  lp_add<kV * kLpVecs>(st, vm, value);
  if (extra >= 0) lp_add<1>(st, xe, [&](int) { return xe; });
  float bound = INFINITY;
  if (top > 0) {
    constexpr int kLanes = kLpThreads / kLpGroups;   // neighbouring lanes form a group
    float g = fmaxf(vm, xe);
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) g = fmaxf(g, __shfl_xor_sync(0xFFFFFFFFu, g, o));
    if (tid % kLanes == 0) sm.gmax[tid / kLanes] = g;
    __syncthreads();
    if (tid < kLpGroups) raise_bound(sm.gmax[tid], kLpGroups / 4);
    __syncthreads();
    // -inf is no bound: what is above it is collected, the rest if that is too little
    bound = fmaxf(sm.bound, -3.4028235e38f);
    push_from(v0, bound);
    if (extra >= 0 && xe >= bound) lp_push(sm, xe, extra);
  }
  // ---- the rest of the slice. The bound is renewed before the fourth chunk
  // and then whenever three times as many have been read, from the candidates
  // so far: 64 groups of them give one that about `top` reach, however many
  // there are. (1024 x 151936 bf16, top 5 / 20 / 32: 66 / 80 / 85 us; with
  // renewals five times as far apart and only while the candidates were 128
  // at most 72 / 104 / 544, the last by the path for full buffers.)
  int renew = v0 + 3 * kStep;
  if (top == 0 || renew + kStep > v1) renew = INT_MAX;
  for (int base = v0 + kStep, slot = 0; base < v1; base += kStep, slot ^= 1) {
    if constexpr (kAhead) fetch(base + kStep, slot ^ 1);
    if (base + kStep > v1) {
      load(base);
    } else if constexpr (kAhead) {
      cp_async_wait<1>();
#pragma unroll
      for (int j = 0; j < kLpVecs; ++j) v[j] = ring[(slot * kLpVecs + j) * kLpThreads + tid];
    } else {
      load_full(base);
    }
    if (base >= renew) {
      renew = base + 2 * (base - v0);
      if (renew + kStep > v1) renew = INT_MAX;
      __syncthreads();
      const int c = sm.count;
      if (c >= top && c <= kLpCap) {
        if (tid < kLpGroups) {
          float g = -INFINITY;
          for (int k = tid; k < c; k += kLpGroups) g = fmaxf(g, lp_value(sm.buf[k]));
          sm.gmax[tid] = g;
        }
        __syncthreads();
        if (tid < min(c, kLpGroups)) raise_bound(sm.gmax[tid], (min(c, kLpGroups) + 3) / 4);
      }
      __syncthreads();
      bound = fmaxf(bound, sm.bound);
    }
    vm = chunk_max();
    lp_add<kV * kLpVecs>(st, vm, value);
    if (vm >= bound) push_from(base, bound);
  }
  // ---- statistics of the CTA: lanes, then warps in order
  st.warp_join();
  if (lane == 0) sm.wst[warp] = st;
  __syncthreads();
  if (warp == 0) {
    st.init();
    if (lane < kLpThreads / 32) st = sm.wst[lane];
    st.warp_join();
    if (lane == 0) sm.st = st;
  }
  // ---- alternatives of the slice
  if (top > 0) {
    int c = sm.count;
    if (c > kLpCap || c < min(top, slice_n)) {
      // Once more, with keys: the buffer is cut back to the best `top`
      // whenever the next round might not fit.
      constexpr int kRound = kLpCap / 2;   // elements a round can add
      const int lo = rank == 0 ? 0 : head + v0 * kV;
      const int hi = rank == cs - 1 ? p.vocab : head + v1 * kV;
      uint64_t cut = 0;
      __syncthreads();
      if (tid == 0) sm.count = 0;
      __syncthreads();
      for (int base = lo; base < hi; base += kRound) {
        for (int i = base + tid; i < min(hi, base + kRound); i += kLpThreads) {
          const float w = lp_to_f32(x[i]);
          if (lp_key(w, i) > cut) lp_push(sm, w, i);
        }
        __syncthreads();
        c = sm.count;
        __syncthreads();
        if (c > kLpCap - kRound) {
          lp_select<kLpThreads>(sm, c, top);
          c = sm.n_best;
          cut = c == top ? sm.best[top - 1] : 0;
          if (tid < c) sm.buf[tid] = sm.best[tid];
          if (tid == 0) sm.count = c;
          __syncthreads();
        }
      }
    }
    lp_select<kLpThreads>(sm, c, top);
  } else {
    __syncthreads();
  }
  // ---- the cluster's slices meet in the first CTA
  if (cs > 1) {
    __syncthreads();   // the slice's results are there
    cluster_wait();
    LpSmem* o = cl.map_shared_rank(&sm, 0);
    if (tid == 0) {
      o->cst[rank] = sm.st;
      o->cn[rank] = top > 0 ? sm.n_best : 0;
    }
    if (top > 0 && tid < sm.n_best) o->cbest[rank][tid] = sm.best[tid];
    cluster_arrive();
    cluster_wait();
    if (rank != 0) return;
    if (warp == 0) {
      st.init();
      if (lane < cs) st = sm.cst[lane];
      st.warp_join();
      if (lane == 0) sm.st = st;
    }
    if (top > 0) {
      int c = 0;
      for (int r = 0; r < cs; ++r) {
        const int n = sm.cn[r];
        if (tid < n) sm.buf[c + tid] = sm.cbest[r][tid];
        c += n;
      }
      __syncthreads();
      lp_select<kLpThreads>(sm, c, top);
    }
  }
  __syncthreads();
  const LpStats a = sm.st;
  const float logs = logf(a.s);
  if (tid == 0) {
    if (p.logprob) p.logprob[row] = (x_token - a.m) - logs;   // NaN for no token
    if (p.entropy) p.entropy[row] = logs - a.t / a.s;
  }
  if (tid < top) {
    const uint64_t key = sm.best[tid];
    const int64_t at = static_cast<int64_t>(row) * top + tid;
    if (p.top_ids) p.top_ids[at] = lp_index(key);
    if (p.top_logprobs) p.top_logprobs[at] = (lp_value(key) - a.m) - logs;
  }
}

template <typename T, int kLpThreads>
dfv_status logprob_launch_t(const LogprobParams& p, int rows, int cs, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(rows) * cs);
  cfg.blockDim = dim3(kLpThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cs;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, logprob_kernel<T, kLpThreads>, p) == cudaSuccess ? DFV_OK
                                                                                   : DFV_ERR_CUDA;
}

// Up to two rows an SM (64 if they are short): CTAs of 1024 threads, one to an
// SM, for few rows as many to a row as leave a round of loads per slice (a
// cluster of more than eight lies in one GPC, so only for a handful of rows).
// More: CTAs of 128 threads, eight to an SM (seven with 16-bit rows, for their
// shared memory); a row is split where that fills the last wave better. A
// CTA's start and end cost about as much as a twentieth of a 152 K row beside
// its share, with alternatives more the more there are. (bf16, 151936 logits,
// top 8, us, by 1024 / 128 threads: 100 rows 13 / 18, 300 rows 26 / 39, 1024
// rows 93 / 67; 100 rows of 5000 4.5 / 7.0, 300 rows of 1000 9.3 / 6.4.)
template <typename T>
dfv_status logprob_launch(const LogprobParams& p, int rows, cudaStream_t stream) {
  const int sms = sm_count();
  if (rows <= 64 || (rows <= 2 * sms && p.vocab >= 4096)) {
    const int round = 1024 * kLpVecs * LpVec<T>::kN;
    const int most = rows <= 4 ? 16 : rows <= 16 ? 8 : rows <= 32 ? 4 : rows <= 64 ? 2 : 1;
    int cs = 1;
    while (cs < most && p.vocab > cs * round) cs <<= 1;
    if (cs == 16) {
      static std::atomic<int> allowed[64];   // clusters above eight need leave, once per device
      int dev = 0;
      if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return DFV_ERR_CUDA;
      if (!allowed[dev].load(std::memory_order_acquire)) {
        if (cudaFuncSetAttribute(logprob_kernel<T, 1024>,
                                 cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
          return DFV_ERR_CUDA;
        allowed[dev].store(1, std::memory_order_release);
      }
    }
    return logprob_launch_t<T, 1024>(p, rows, cs, stream);
  }
  const int64_t slots = static_cast<int64_t>(sms) * (sizeof(T) == 2 ? 7 : 8);
  const double start = p.top > 0 ? 0.12 + 0.006 * p.top : 0.05;
  int cs = 1;
  double best = 1e30;
  for (int c = 1; c <= 8; c <<= 1) {
    const double cost = ((rows * static_cast<int64_t>(c) + slots - 1) / slots) * (1.0 / c + start);
    if (cost < best) {
      best = cost;
      cs = c;
    }
  }
  return logprob_launch_t<T, 128>(p, rows, cs, stream);
}

}  // namespace dfv

extern "C" dfv_status dfv_token_logprobs(int n_rows, int vocab, int logits_dtype,
                                         const void* logits, int64_t stride_row,
                                         const int32_t* tokens, int top, float* logprob,
                                         float* entropy, int32_t* top_ids, float* top_logprobs,
                                         uint32_t* status, dfv_stream_t stream) {
  using namespace dfv;
  if (logits_dtype != DFV_DTYPE_F32 && logits_dtype != DFV_DTYPE_BF16) return DFV_ERR_UNSUPPORTED;
  const size_t size = logits_dtype == DFV_DTYPE_F32 ? 4 : 2;
  if (n_rows < 0 || n_rows > (1 << 27) || vocab < 1 || vocab > (1 << 30) || top < 0 ||
      top > DFV_MAX_TOP || top > vocab || (n_rows > 1 && stride_row < vocab))
    return DFV_ERR_INVALID;
  if (n_rows == 0) return DFV_OK;
  if (!logits || !aligned(logits, size) || (logprob && !tokens)) return DFV_ERR_INVALID;
  if (top > 0 && !top_ids && !top_logprobs) return DFV_ERR_INVALID;
  LogprobParams p = {vocab, top, logits, stride_row, tokens, logprob, entropy, top_ids,
                     top_logprobs, status};
  return logits_dtype == DFV_DTYPE_F32
             ? logprob_launch<float>(p, n_rows, static_cast<cudaStream_t>(stream))
             : logprob_launch<__nv_bfloat16>(p, n_rows, static_cast<cudaStream_t>(stream));
}
