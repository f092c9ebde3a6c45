// A token from each row of logits by temperature, top-k, top-p and min-p, from
// one given random number; over a draft tree also the walk along the children
// that were drawn.
//
//   w_i = exp((x_i - max x) / T)
//   top-k  the k largest x (ties to the lowest index); Z = sum of their w
//   top-p  of these, in that order, the shortest run whose w reach p Z
//   min-p  of these, w_i >= max(min_p, 2^-40)
//   token  the first index, in index order, at which the running sum of the
//          kept w exceeds u times their total
//
// The token is a whole number, so its borders have to be exact far beyond
// float32: with 150 K tokens and sums that are off by 2^-24 one row in a
// hundred would get its neighbour. Weights therefore are 64-bit integers in
// units of 2^-44 of a power of two above the largest: 2^t by a table of
// 2^(j/64) in 32 bits and a cubic for the rest, t = (x - base) log2(e) / T in
// two floats (off by about 2^-31 of the weight). Sums of integers have no order, so every
// pass over the row agrees with every other and nothing depends on how the row
// is split.
//
// A row belongs to a cluster of 1 to 16 CTAs that keep it in shared memory:
// it is read from memory once, and passes over it run at shared memory's rate.
// The first CTA decides, the others carry out what it asks for. Passes:
//
//   1. maximum, while the row arrives;
//   2. the sum of all weights; tokens within 2^-12 of the largest go to a list.
//      If the list holds both cuts (a model that is reasonably sure), it is
//      sorted in the first CTA and the token comes from it;
//   3. otherwise counts and weights of 1024 bins of the logit, the bin with the
//      cut, its tokens sorted (a bin of more than 512 is cut by its keys'
//      bits; equal keys are counted in index order);
//   4. the sum of the kept weights per warp, and the warp with the token once
//      more.
//
// Without top-k and top-p pass 2 is pass 4.

#include <atomic>
#include <climits>

#include "common.cuh"

namespace dfv {

constexpr int kSmpThreads = 512;
constexpr int kSmpWarps = kSmpThreads / 32;
constexpr int kSmpBins = 1024;
constexpr int kSmpList = kSmpThreads;      // one sorted token a thread
constexpr int kSmpMaxCluster = 16;
constexpr int kSmpMaxVocab = 1 << 19;      // sums of weights stay below 2^63
constexpr float kSmpMinT = 0x1p-100f;      // below: greedy

struct SampleParams {
  int n_rows, vocab;
  const void* logits;
  int64_t stride;
  const float* uniform;
  dfv_sampling s;
  int32_t* token;
  float* logprob;
  uint32_t* status;
  // the walk (parent null: none)
  const int32_t *parent, *tokens;
  int32_t *accept_len, *path, *out_tokens;
  unsigned int* ticket;
  int slice_vecs;    // 16-byte vectors of shared memory for the slice
};

// round(2^(31 + j / 64))
__constant__ uint32_t kSmpExp2[64] = {
    0x80000000u, 0x8164D1F4u, 0x82CD8699u, 0x843A28C4u, 0x85AAC368u, 0x871F6197u, 0x88980E81u, 0x8A14D575u,
    0x8B95C1E4u, 0x8D1ADF5Bu, 0x8EA4398Bu, 0x9031DC43u, 0x91C3D374u, 0x935A2B2Fu, 0x94F4EFA9u, 0x96942D37u,
    0x9837F052u, 0x99E04593u, 0x9B8D39BAu, 0x9D3ED9A7u, 0x9EF53261u, 0xA0B05110u, 0xA2704303u, 0xA43515AEu,
    0xA5FED6AAu, 0xA7CD93B5u, 0xA9A15AB5u, 0xAB7A39B6u, 0xAD583EEAu, 0xAF3B78ADu, 0xB123F582u, 0xB311C413u,
    0xB504F334u, 0xB6FD91E3u, 0xB8FBAF47u, 0xBAFF5AB2u, 0xBD08A39Fu, 0xBF1799B6u, 0xC12C4CCAu, 0xC346CCDAu,
    0xC5672A11u, 0xC78D74C9u, 0xC9B9BD86u, 0xCBEC14FFu, 0xCE248C15u, 0xD06333DBu, 0xD2A81D92u, 0xD4F35AACu,
    0xD744FCCBu, 0xD99D15C2u, 0xDBFBB798u, 0xDE60F482u, 0xE0CCDEECu, 0xE33F8973u, 0xE5B906E7u, 0xE8396A50u,
    0xEAC0C6E8u, 0xED4F301Fu, 0xEFE4B99Cu, 0xF281773Cu, 0xF5257D15u, 0xF7D0DF73u, 0xFA83B2DBu, 0xFD3E0C0Du,
};

enum SmpState {
  kStart, kAfterHist, kAfterRange, kAfterKeyHist, kAfterCount, kAfterFind, kAfterGather, kAfterSum
};

enum SmpOp {
  kOpDone, kOpHistLogit, kOpGatherLogit, kOpRangeLogit, kOpHistKey, kOpGatherKey, kOpCountEqual,
  kOpFindEqual, kOpSum, kOpPick
};

struct SmpCmd {
  int op, bin, shift, rank, warp, nth;
  uint32_t khi, klo;     // keys, both included
  uint64_t target, total;
};

struct SmpSmem {
  uint32_t cnt[kSmpBins], mlo[kSmpBins], mhi[kSmpBins];   // a bin's count and weight
  uint64_t buf[kSmpList];      // this CTA's list
  uint64_t keys[kSmpList];     // first CTA: the cluster's
  uint64_t sorted[kSmpList], run[kSmpList];   // in order, and running weights
  uint32_t table[64];
  uint64_t wtot[2][kSmpWarps];
  float wmax[kSmpWarps];
  float xmax[kSmpMaxCluster];
  // first CTA: what the others report
  uint64_t xsum[kSmpMaxCluster * kSmpWarps];
  uint32_t xcnt[kSmpMaxCluster * kSmpWarps];
  int xlist[kSmpMaxCluster];
  uint32_t xlo[kSmpMaxCluster], xhi[kSmpMaxCluster];
  uint32_t found;
  // parameters of the row
  float t_inv_hi, t_inv_lo, temperature, top_p, min_p, u;
  double ln_min;
  int top_k, bad;
  int list_n;
  uint32_t lo, hi, first;
  SmpCmd cmd;
  // first CTA: a search, its hit, and the cut so far with the weight up to it
  bool by_mass;
  int hit;
  uint32_t hit_cnt;
  uint64_t target, acc_cnt, acc_mass, need, mass;
  uint32_t cut_key;
  int cut_index;
  float result_logprob;
  int result;
};

__device__ __forceinline__ uint32_t smp_order(float x) {   // -0 equals +0
  const uint32_t u = __float_as_uint(x + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float smp_value(uint32_t o) {
  return __uint_as_float((o & 0x80000000u) ? (o & 0x7FFFFFFFu) : ~o);
}
__device__ __forceinline__ float smp_max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

template <typename T> struct SmpVec;
template <> struct SmpVec<float> {
  static constexpr int kN = 4;
  static __device__ __forceinline__ float at(const uint4& v, int i) {
    return __uint_as_float(i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w);
  }
  static __device__ __forceinline__ float low() { return -INFINITY; }
};
template <> struct SmpVec<__nv_bfloat16> {
  static constexpr int kN = 8;
  static __device__ __forceinline__ float at(const uint4& v, int i) {
    const uint32_t w = i < 2 ? v.x : i < 4 ? v.y : i < 6 ? v.z : v.w;
    return __uint_as_float(i & 1 ? w & 0xFFFF0000u : w << 16);
  }
  static __device__ __forceinline__ __nv_bfloat16 low() { return __float2bfloat16(-INFINITY); }
};

// Cluster barrier, and addresses of the same variable in another CTA.
__device__ __forceinline__ void smp_cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
}
__device__ __forceinline__ void smp_cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ void smp_cluster_sync() {
  smp_cluster_arrive();
  smp_cluster_wait();
}
template <typename V>
__device__ __forceinline__ V* smp_remote(V* p, int rank) {
  uint64_t out;
  asm volatile("mapa.u64 %0, %1, %2;" : "=l"(out) : "l"(p), "r"(rank));
  return reinterpret_cast<V*>(out);
}

__device__ __forceinline__ uint64_t smp_warp_sum(uint64_t v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}
__device__ __forceinline__ uint64_t smp_warp_scan(uint64_t v, int lane) {   // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t w = __shfl_up_sync(0xFFFFFFFFu, v, o);
    if (lane >= o) v += w;
  }
  return v;
}

// ln(w / total), as far from 0 as it is where w is nearly all
__device__ __forceinline__ float smp_log_share(uint64_t w, uint64_t total) {
  return w > total / 2 ? log1pf(-static_cast<float>(total - w) / static_cast<float>(total))
                       : logf(static_cast<float>(w) / static_cast<float>(total));
}

// The walk from the root along the lowest-index child whose token is the one
// drawn for its parent (one warp; the same rule as the greedy walk).
__device__ void smp_walk(const SampleParams& p, int lane) {
  int par[3], tok[3], drawn[3];
  bool bad = false;
#pragma unroll
  for (int s = 0; s < 3; ++s) {
    const int i = lane + 32 * s;
    par[s] = -2;
    tok[s] = drawn[s] = 0;
    if (i < p.n_rows) drawn[s] = __ldcg(p.token + i);   // written by other SMs
    if (i >= 1 && i < p.n_rows) {
      par[s] = p.parent[i];
      tok[s] = p.tokens[i];
      if (par[s] < 0 || par[s] >= i) {
        bad = true;
        par[s] = 0;
      }
    }
  }
  if (__any_sync(0xFFFFFFFFu, bad) && lane == 0) report(p.status, DFV_DEV_BAD_TREE);
  auto of = [&](const int* v, int i) {
    const int a = __shfl_sync(0xFFFFFFFFu, v[0], i & 31);
    const int b = __shfl_sync(0xFFFFFFFFu, v[1], i & 31);
    const int c = __shfl_sync(0xFFFFFFFFu, v[2], i & 31);
    return i < 32 ? a : i < 64 ? b : c;
  };
  int cur = 0, len = 0;
  while (true) {
    const int t = of(drawn, cur);
    const unsigned b0 = __ballot_sync(0xFFFFFFFFu, par[0] == cur && tok[0] == t);
    const unsigned b1 = __ballot_sync(0xFFFFFFFFu, par[1] == cur && tok[1] == t);
    const unsigned b2 = __ballot_sync(0xFFFFFFFFu, par[2] == cur && tok[2] == t);
    const int next = b0 ? __ffs(b0) - 1 : b1 ? 31 + __ffs(b1) : b2 ? 63 + __ffs(b2) : -1;
    if (lane == 0) {
      p.path[len] = cur;
      p.out_tokens[len] = t;   // the child's token is the one drawn
    }
    ++len;
    if (next < 0 || t < 0 || len >= p.n_rows) break;   // t < 0: none was drawn here
    cur = next;
  }
  for (int i = len + lane; i < p.n_rows; i += 32) p.path[i] = p.out_tokens[i] = -1;
  if (lane == 0) *p.accept_len = len;
}

// One warp, all lanes: the row's result; the last row's warp walks.
__device__ void smp_finish(const SampleParams& p, int row, int token, float logprob, int lane) {
  unsigned last = 0;
  if (lane == 0) {
    p.token[row] = token;
    if (p.logprob) p.logprob[row] = logprob;
    if (p.parent) {
      __threadfence();
      last = atomicAdd(p.ticket, 1u) == static_cast<unsigned>(p.n_rows) - 1;
      if (last) {
        *p.ticket = 0u;   // ready for the next launch
        __threadfence();
      }
    }
  }
  if (__shfl_sync(0xFFFFFFFFu, last, 0)) smp_walk(p, lane);
}

template <typename T>
__global__ void __launch_bounds__(kSmpThreads, 2)
    sample_kernel(const __grid_constant__ SampleParams p) {
  extern __shared__ __align__(128) uint8_t smem_raw[];
  SmpSmem& sm = *reinterpret_cast<SmpSmem*>(smem_raw);
  uint4* xs = reinterpret_cast<uint4*>(smem_raw + ((sizeof(SmpSmem) + 127) / 128) * 128);
  constexpr int kV = SmpVec<T>::kN;
  int cs, rank;
  asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(cs));
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  const int row = blockIdx.x / cs, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  smp_cluster_arrive();   // waited for before another CTA's memory is touched
  if (tid < 64) sm.table[tid] = kSmpExp2[tid];
  if (tid == 0) sm.list_n = 0;
  grid_dep_wait();
  grid_dep_launch_dependents();   // (after the wait: see common.cuh)

  // ---- the row: a head before the first 16-byte boundary, whole vectors, a
  // tail. Vectors are dealt in equal runs; the first CTA has the head too, the
  // last one the tail. A slice starts with a whole vector of shared memory,
  // padded with -inf.
  const T* x = static_cast<const T*>(p.logits) + row * p.stride;
  const int over = static_cast<int>(reinterpret_cast<uintptr_t>(x) & 15);
  const int head = min(p.vocab, (16 - over) % 16 / static_cast<int>(sizeof(T)));
  const int nv = (p.vocab - head) / kV;
  const int v0 = static_cast<int>(static_cast<int64_t>(nv) * rank / cs);
  const int v1 = static_cast<int>(static_cast<int64_t>(nv) * (rank + 1) / cs);
  const int at0 = rank == 0 && head > 0 ? 1 : 0;           // slice vectors before v0
  const int tail = rank == cs - 1 ? p.vocab - head - nv * kV : 0;
  const int n_vecs = at0 + (v1 - v0) + (tail > 0 ? 1 : 0);
  const int first = head + (v0 - at0) * kV;                // row index of the slice's element 0
  for (int i = tid; i < v1 - v0; i += kSmpThreads)
    cp_async16(&xs[at0 + i], reinterpret_cast<const uint4*>(x + head) + v0 + i);
  T* xe = reinterpret_cast<T*>(xs);
  if (at0 && tid < kV) xe[tid] = first + tid >= 0 ? x[first + tid] : SmpVec<T>::low();
  if (tail > 0 && tid >= 32 && tid < 32 + kV) {
    const int i = tid - 32;
    xe[(n_vecs - 1) * kV + i] = i < tail ? x[head + nv * kV + i] : SmpVec<T>::low();
  }
  if (tid == kSmpThreads - 1) {
    // the row's parameters, meanwhile
    const float temp = p.s.temperature ? p.s.temperature[row] : p.s.temperature_all;
    const float top_p = p.s.top_p ? p.s.top_p[row] : p.s.top_p_all;
    const float min_p = p.s.min_p ? p.s.min_p[row] : p.s.min_p_all;
    const float u = p.uniform[row];
    sm.bad = !(temp >= 0.0f) || temp == INFINITY || top_p != top_p || min_p != min_p ||
             !(u >= 0.0f && u < 1.0f);
    const double inv = 1.4426950408889634074 / static_cast<double>(temp);
    sm.t_inv_hi = static_cast<float>(inv);
    sm.t_inv_lo = static_cast<float>(inv - static_cast<double>(sm.t_inv_hi));
    sm.temperature = temp;
    sm.top_p = top_p;
    sm.min_p = fminf(min_p, 1.0f);
    sm.u = u;
    sm.top_k = p.s.top_k ? p.s.top_k[row] : p.s.top_k_all;
    // ln(max(min_p, 2^-40))
    sm.ln_min = sm.min_p > 0x1p-40f ? log(static_cast<double>(sm.min_p)) : -27.725887222397812377;
  }
  cp_async_wait_all();

  // ---- pass 1: the maximum (each thread over the vectors it copied)
  float mx = -INFINITY;
  for (int i = tid; i < v1 - v0; i += kSmpThreads) {
    const uint4 v = xs[at0 + i];
#pragma unroll
    for (int e = 0; e < kV; ++e) mx = smp_max_nan(mx, SmpVec<T>::at(v, e));
  }
  __syncthreads();   // the ends of the slice, the parameters
  if (at0 && tid == 0) {
#pragma unroll
    for (int e = 0; e < kV; ++e) mx = smp_max_nan(mx, SmpVec<T>::at(xs[0], e));
  }
  if (tail > 0 && tid == 0) {
#pragma unroll
    for (int e = 0; e < kV; ++e) mx = smp_max_nan(mx, SmpVec<T>::at(xs[n_vecs - 1], e));
  }
  asm volatile("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(mx) : "f"(mx));
  if (lane == 0) sm.wmax[warp] = mx;
  __syncthreads();
  smp_cluster_wait();   // every CTA has started
  if (tid < cs) {
    float a = sm.wmax[0];
#pragma unroll
    for (int i = 1; i < kSmpWarps; ++i) a = smp_max_nan(a, sm.wmax[i]);
    *smp_remote(&sm.xmax[rank], tid) = a;
  }
  smp_cluster_sync();
  float m = sm.xmax[0];
  for (int i = 1; i < cs; ++i) m = smp_max_nan(m, sm.xmax[i]);

  // ---- rows that have no distribution, and greedy ones
  if (!(fabsf(m) < INFINITY) || sm.bad) {
    if (rank == 0 && warp == 0) {
      if (lane == 0) report(p.status, sm.bad ? DFV_DEV_BAD_SAMPLING : DFV_DEV_NONFINITE);
      smp_finish(p, row, -1, NAN, lane);
    }
    return;
  }
  // Vectors of a warp are neighbours, so that warps are in index order.
  const int per = (n_vecs + kSmpWarps - 1) / kSmpWarps;
  const int wv0 = min(n_vecs, warp * per), wv1 = min(n_vecs, wv0 + per);
  if (sm.temperature < kSmpMinT) {
    uint32_t best = 0xFFFFFFFFu;
    for (int v = wv0 + lane; v < wv1; v += 32) {
      const uint4 r = xs[v];
#pragma unroll
      for (int e = 0; e < kV; ++e)
        if (SmpVec<T>::at(r, e) == m)
          best = min(best, static_cast<uint32_t>(first + v * kV + e));
    }
    best = __reduce_min_sync(0xFFFFFFFFu, best);
    if (lane == 0) *smp_remote(&sm.xcnt[rank * kSmpWarps + warp], 0) = best;
    smp_cluster_sync();
    if (rank == 0 && warp == 0) {
      best = 0xFFFFFFFFu;
      for (int i = lane; i < cs * kSmpWarps; i += 32) best = min(best, sm.xcnt[i]);
      best = __reduce_min_sync(0xFFFFFFFFu, best);
      smp_finish(p, row, static_cast<int>(best), 0.0f, lane);
    }
    return;
  }

  // ---- weights. |m| / T up to 2^12: t = x / T log2(e) itself, to 2^-36; above,
  // tokens that count lie so near the maximum that x - m is exact.
  const float chi = sm.t_inv_hi, clo = sm.t_inv_lo, temp = sm.temperature;
  const float base = fabsf(m) * chi <= 4096.0f ? 0.0f : m;
  constexpr float kMagic = 12582912.0f;   // 1.5 * 2^23: the sum's low bits are the integer
  auto split = [&](float v, int& ki) {    // 64 t = ki + 64 r
    const float d = v - base;
    const float th = d * chi;
    const float tl = fmaf(d, clo, fmaf(d, chi, -th));
    const float k = fmaf(th, 64.0f, kMagic);
    ki = __float_as_int(k) - 0x4B400000;
    return fmaf(k - kMagic, -0.015625f, th) + tl;
  };
  int km;
  split(m, km);
  const int top = (km >> 6) + 1;   // the largest weight is in [2^43, 2^44]
  auto weight = [&](float v) -> uint64_t {
    int ki;
    const float r = split(v, ki);
    const uint32_t tj = sm.table[ki & 63];
    // 2^31 (2^r - 1), |r| <= 2^-7: ln2, ln2^2 / 2, ln2^3 / 6; the next term is below 2^-34
    const float q =
        r * fmaf(r, fmaf(r, 0.055504109f * 0x1p31f, 0.24022651f * 0x1p31f), 0.69314718f * 0x1p31f);
    const float tf = __uint_as_float(0x3F800000u | ((tj >> 8) & 0x7FFFFFu));
    const uint32_t f = tj + static_cast<uint32_t>(__float2int_rn(tf * q));
    // f 2^(13 - s), s = top - (ki >> 6) at least 1
    const int s = min(max(top - (ki >> 6), 0) + 19, 63);
    return (static_cast<uint64_t>(f) << 32) >> s;
  };
  // below: no weight left of 2^-44; within 2^-12 of the largest; kept by min-p
  // (finite, so that -inf is below all three)
  const float tau_w = fmaxf(m - 43.0f * 0.69314718f * temp, -3.4028235e38f);
  const float tau_l = fmaxf(m - 12.0f * 0.69314718f * temp, -3.4028235e38f);
  float tau_0;
  {
    const double t0 = static_cast<double>(m) + static_cast<double>(temp) * sm.ln_min;
    tau_0 = __double2float_ru(t0);
  }
  const float bin_scale = (kSmpBins - 0.5f) / (43.0f * 0.69314718f) / temp;
  auto logit_bin = [&](float v) {   // monotone: each operation is
    return min(static_cast<int>((m - v) * bin_scale), kSmpBins - 1);
  };
  const bool by_k = sm.top_k > 0 && sm.top_k < p.vocab, by_p = sm.top_p < 1.0f;

  auto each = [&](auto f) {   // f(value, row index) over this warp's vectors
    for (int v = wv0 + lane; v < wv1; v += 32) {
      const uint4 r = xs[v];
#pragma unroll
      for (int e = 0; e < kV; ++e) f(SmpVec<T>::at(r, e), first + v * kV + e);
    }
  };
  auto key_of = [&](float v, int i) {
    return (static_cast<uint64_t>(smp_order(v)) << 32) | static_cast<uint32_t>(~i);
  };
  auto push = [&](float v, int i) {
    const int k = atomicAdd(&sm.list_n, 1);
    if (k < kSmpList) sm.buf[k] = key_of(v, i);
  };
  auto tell_sum = [&](uint64_t s) {
    s = smp_warp_sum(s);
    if (lane == 0) *smp_remote(&sm.xsum[rank * kSmpWarps + warp], 0) = s;
  };

  // ---- pass 2
  {
    uint64_t s = 0;
    if (!by_k && !by_p) {
      each([&](float v, int) { s += v >= tau_0 ? weight(v) : 0; });
    } else {
      each([&](float v, int i) {
        s += v >= tau_w ? weight(v) : 0;
        if (v >= tau_l) push(v, i);
      });
      __syncthreads();
      if (tid == 0) *smp_remote(&sm.xlist[rank], 0) = sm.list_n;
    }
    tell_sum(s);
  }
  smp_cluster_sync();

  auto hist_add = [&](int b, float v) {
    const uint64_t w = weight(v);
    atomicAdd(&sm.cnt[b], 1u);
    const uint32_t lo = static_cast<uint32_t>(w);
    const uint32_t was = atomicAdd(&sm.mlo[b], lo);
    const uint32_t hi = static_cast<uint32_t>(w >> 32) + (was + lo < was ? 1u : 0u);
    if (hi) atomicAdd(&sm.mhi[b], hi);
  };
  // kept: above the cut, or at it up to an index
  auto kept = [&](const SmpCmd& c, float v, int i) {
    const uint32_t o = smp_order(v);
    return v >= tau_0 && (o > c.khi || (o == c.khi && i <= c.nth));
  };

  // What the first CTA asks for, carried out by all.
  auto carry_out = [&](const SmpCmd& c) {
    switch (c.op) {
      case kOpHistLogit:
      case kOpHistKey:
        for (int b = tid; b < kSmpBins; b += kSmpThreads) sm.cnt[b] = sm.mlo[b] = sm.mhi[b] = 0;
        __syncthreads();
        if (c.op == kOpHistLogit) {
          each([&](float v, int) {
            if (v >= tau_w) hist_add(logit_bin(v), v);
          });
        } else {
          each([&](float v, int) {
            const uint32_t o = smp_order(v);
            if (o <= c.khi && o >= c.klo) hist_add((c.khi - o) >> c.shift, v);
          });
        }
        break;
      case kOpGatherLogit:
      case kOpGatherKey:
        if (tid == 0) sm.list_n = 0;
        __syncthreads();
        if (c.op == kOpGatherLogit) {
          each([&](float v, int i) {
            if (v >= tau_w && logit_bin(v) == c.bin) push(v, i);
          });
        } else {
          each([&](float v, int i) {
            const uint32_t o = smp_order(v);
            if (o <= c.khi && o >= c.klo) push(v, i);
          });
        }
        __syncthreads();
        if (tid == 0) *smp_remote(&sm.xlist[rank], 0) = sm.list_n;
        break;
      case kOpRangeLogit: {
        uint32_t lo = 0xFFFFFFFFu, hi = 0;
        if (tid == 0) {
          sm.lo = lo;
          sm.hi = hi;
        }
        __syncthreads();
        each([&](float v, int) {
          if (v >= tau_w && logit_bin(v) == c.bin) {
            lo = min(lo, smp_order(v));
            hi = max(hi, smp_order(v));
          }
        });
        lo = __reduce_min_sync(0xFFFFFFFFu, lo);
        hi = __reduce_max_sync(0xFFFFFFFFu, hi);
        if (lane == 0) {
          atomicMin(&sm.lo, lo);
          atomicMax(&sm.hi, hi);
        }
        __syncthreads();
        if (tid == 0) {
          *smp_remote(&sm.xlo[rank], 0) = sm.lo;
          *smp_remote(&sm.xhi[rank], 0) = sm.hi;
        }
        break;
      }
      case kOpCountEqual: {
        uint32_t n = 0;
        each([&](float v, int) { n += smp_order(v) == c.khi; });
        n = __reduce_add_sync(0xFFFFFFFFu, n);
        if (lane == 0) *smp_remote(&sm.xcnt[rank * kSmpWarps + warp], 0) = n;
        break;
      }
      case kOpFindEqual:   // the nth of a warp's equal keys
        if (rank == c.rank && warp == c.warp) {
          int before = 0;
          for (int v = wv0; v < wv1; v += 32) {
            int n = 0;
            uint4 r = make_uint4(0, 0, 0, 0);
            if (v + lane < wv1) {
              r = xs[v + lane];
#pragma unroll
              for (int e = 0; e < kV; ++e) n += smp_order(SmpVec<T>::at(r, e)) == c.khi;
            }
            int at = before + static_cast<int>(smp_warp_scan(static_cast<uint64_t>(n), lane)) - n;
            if (at <= c.nth && c.nth < at + n) {
#pragma unroll
              for (int e = 0; e < kV; ++e) {
                if (smp_order(SmpVec<T>::at(r, e)) != c.khi) continue;
                if (at++ == c.nth)
                  *smp_remote(&sm.found, 0) = static_cast<uint32_t>(first + (v + lane) * kV + e);
              }
            }
            before += __reduce_add_sync(0xFFFFFFFFu, n);
          }
        }
        break;
      case kOpSum: {
        uint64_t s = 0;
        each([&](float v, int i) { s += kept(c, v, i) ? weight(v) : 0; });
        tell_sum(s);
        break;
      }
      case kOpPick:   // the token in this warp's run at which its sum exceeds the target
        if (rank == c.rank && warp == c.warp) {
          uint64_t before = 0;
          int token = -1;
          float logprob = 0.0f;
          for (int v = wv0; v < wv1; v += 32) {
            uint64_t s = 0;
            uint4 r = make_uint4(0, 0, 0, 0);
            const int i0 = first + (v + lane) * kV;
            if (v + lane < wv1) {
              r = xs[v + lane];
#pragma unroll
              for (int e = 0; e < kV; ++e) {
                const float z = SmpVec<T>::at(r, e);
                s += kept(c, z, i0 + e) ? weight(z) : 0;
              }
            }
            const uint64_t incl = before + smp_warp_scan(s, lane);
            const bool mine = incl - s <= c.target && c.target < incl;
            const unsigned who = __ballot_sync(0xFFFFFFFFu, mine);
            if (who) {
              if (mine) {
                uint64_t at = incl - s;
#pragma unroll 1
                for (int e = 0; e < kV; ++e) {
                  const float z = SmpVec<T>::at(r, e);
                  const uint64_t w = kept(c, z, i0 + e) ? weight(z) : 0;
                  if (token < 0 && c.target < at + w) {
                    token = i0 + e;
                    logprob = smp_log_share(w, c.total);
                  }
                  at += w;
                }
              }
              token = __shfl_sync(0xFFFFFFFFu, token, __ffs(who) - 1);
              logprob = __shfl_sync(0xFFFFFFFFu, logprob, __ffs(who) - 1);
              break;
            }
            before = __shfl_sync(0xFFFFFFFFu, incl, 31);
          }
          smp_finish(p, row, token, logprob, lane);
        }
        break;
      default: break;
    }
  };

  // ---- what the first CTA decides from the reports (all of its threads)
  int state = kStart;
  // Inclusive sums over the CTA's threads of two numbers at once.
  auto block_scan = [&](uint64_t& a, uint64_t& b) {
    a = smp_warp_scan(a, lane);
    b = smp_warp_scan(b, lane);
    __syncthreads();
    if (lane == 31) {
      sm.wtot[0][warp] = a;
      sm.wtot[1][warp] = b;
    }
    __syncthreads();
    for (int i = 0; i < warp; ++i) {
      a += sm.wtot[0][i];
      b += sm.wtot[1][i];
    }
  };
  // The cluster's list (at most kSmpList keys), sorted, with running weights.
  auto collect = [&]() {
    int n = 0, src = 0, off = -1;
    for (int r = 0; r < cs; ++r) {
      const int c = sm.xlist[r];
      if (tid >= n && tid < n + c) {
        src = r;
        off = tid - n;
      }
      n += c;
    }
    const uint64_t key = off >= 0 ? *smp_remote(&sm.buf[off], src) : 0;
    sm.keys[tid] = key;
    sm.run[tid] = 0;
    __syncthreads();
    if (tid < n) {
      int above = 0;
#pragma unroll 8
      for (int i = 0; i < n; ++i) above += sm.keys[i] > key;
      sm.sorted[above] = key;
      sm.run[above] = weight(smp_value(static_cast<uint32_t>(key >> 32)));
    }
    __syncthreads();
    uint64_t a = sm.run[tid], b = 0;
    block_scan(a, b);
    sm.run[tid] = a;
    __syncthreads();
    return n;
  };
  // top_p of `mass`, rounded up, one unit at least
  auto share = [&](uint64_t mass) -> uint64_t {
    if (!(sm.top_p > 0.0f)) return 1;
    const uint64_t f = __float2ull_rz(sm.top_p * 0x1p64f);
    const uint64_t hi = __umul64hi(f, mass) + (f * mass != 0 ? 1 : 0);
    return hi > 0 ? hi : 1;
  };
  // The histograms of all CTAs summed, and the bin in which the running count
  // (weight) from bin 0 on reaches `target`: sm.hit (-1: never), sm.hit_cnt, and
  // what comes before it added to sm.acc_cnt, sm.acc_mass.
  auto locate = [&]() {
    const bool by_mass = sm.by_mass;
    const uint64_t target = sm.target - (by_mass ? sm.acc_mass : sm.acc_cnt);
    uint64_t c2[2], m2[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int b = 2 * tid + k;
      c2[k] = m2[k] = 0;
      for (int r = 0; r < cs; ++r) {
        c2[k] += *smp_remote(&sm.cnt[b], r);
        m2[k] += (static_cast<uint64_t>(*smp_remote(&sm.mhi[b], r)) << 32) +
                 *smp_remote(&sm.mlo[b], r);
      }
    }
    uint64_t a = c2[0] + c2[1], b = m2[0] + m2[1];
    if (tid == 0) sm.hit = -1;
    block_scan(a, b);
    uint64_t ca = a - c2[0] - c2[1], ma = b - m2[0] - m2[1];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint64_t was = by_mass ? ma : ca, now = by_mass ? ma + m2[k] : ca + c2[k];
      if (was < target && target <= now) {   // one thread's, if any
        sm.hit = 2 * tid + k;
        sm.hit_cnt = static_cast<uint32_t>(c2[k]);
        sm.acc_cnt += ca;
        sm.acc_mass += ma;
      }
      ca += c2[k];
      ma += m2[k];
    }
    __syncthreads();
  };
  // Starts the search for the cut at which the running count (weight) of the
  // tokens, from the largest on, reaches `target`.
  auto search = [&](SmpCmd& c, bool by_mass, uint64_t target) {
    __syncthreads();
    if (tid == 0) {
      sm.by_mass = by_mass;
      sm.target = target;
      sm.acc_cnt = sm.acc_mass = 0;
    }
    c.op = kOpHistLogit;
    state = kAfterHist;
  };
  // A list that holds every cut: the token comes from it. False: it does not.
  auto from_list = [&]() {
    int n = 0;
    for (int r = 0; r < cs; ++r) n += min(sm.xlist[r], kSmpList + 1);
    if (n > kSmpList) return false;
    collect();
    int keep = n;
    uint64_t mass = sm.mass;
    if (by_k) {
      if (sm.top_k > n) return false;
      keep = sm.top_k;
      mass = sm.run[keep - 1];
    }
    if (by_p) {
      const uint64_t goal = share(mass);
      if (sm.run[keep - 1] < goal) return false;
      // tokens before which less than the goal has come together
      keep = min(keep,
                 __syncthreads_count(tid < n && (tid == 0 ? 0 : sm.run[tid - 1]) < goal));
    }
    // min-p cuts the same order
    keep = min(keep, __syncthreads_count(
                         tid < n &&
                         smp_value(static_cast<uint32_t>(sm.sorted[tid] >> 32)) >= tau_0));
    const uint64_t total = sm.run[keep - 1];
    const uint64_t target = __umul64hi(__float2ull_rz(sm.u * 0x1p64f), total);
    if (tid < keep) {
      const uint32_t mine = ~static_cast<uint32_t>(sm.sorted[tid]);
      const uint64_t w = sm.run[tid] - (tid == 0 ? 0 : sm.run[tid - 1]);
      uint64_t before = 0, was = 0;
#pragma unroll 4
      for (int i = 0; i < keep; ++i) {
        const uint64_t now = sm.run[i];
        if (~static_cast<uint32_t>(sm.sorted[i]) < mine) before += now - was;
        was = now;
      }
      if (before <= target && target < before + w) {
        sm.result = static_cast<int>(mine);
        sm.result_logprob = smp_log_share(w, total);
      }
    }
    __syncthreads();
    if (warp == 0) smp_finish(p, row, sm.result, sm.result_logprob, lane);
    return true;
  };
  // The total of the warps' sums, and the warp in which they reach u of it.
  auto pick = [&](SmpCmd& c) {
    uint64_t a = tid < cs * kSmpWarps ? sm.xsum[tid] : 0, b = 0;
    const uint64_t mine = a;
    block_scan(a, b);
    uint64_t total = 0;
    for (int i = 0; i < kSmpWarps; ++i) total += sm.wtot[0][i];
    const uint64_t target = __umul64hi(__float2ull_rz(sm.u * 0x1p64f), total);
    if (a - mine <= target && target < a) {
      sm.hit = tid;
      sm.acc_mass = target - (a - mine);
    }
    __syncthreads();
    c.op = kOpPick;
    c.khi = sm.cut_key;
    c.nth = sm.cut_index;
    c.rank = sm.hit / kSmpWarps;
    c.warp = sm.hit % kSmpWarps;
    c.target = sm.acc_mass;
    c.total = total;
  };
  // The next command.
  auto decide = [&](SmpCmd& c) {
    bool refine = false, found = false;
    switch (state) {
      case kStart: {
        uint64_t a = tid < cs * kSmpWarps ? sm.xsum[tid] : 0, b = 0;
        block_scan(a, b);
        if (tid == kSmpThreads - 1) {
          sm.mass = a;            // of all tokens
          sm.cut_key = 0;         // no cut: every key is above it
          sm.cut_index = 0;
        }
        __syncthreads();
        if (!by_k && !by_p) {
          pick(c);
        } else if (from_list()) {
          c.op = kOpDone;
        } else {
          search(c, !by_k, by_k ? static_cast<uint64_t>(sm.top_k) : share(sm.mass));
        }
        return;
      }
      case kAfterHist:
        locate();
        if (sm.hit < 0) {   // fewer than top_k tokens have a weight
          found = true;
          break;
        }
        c.bin = sm.hit;
        c.op = sm.hit_cnt <= kSmpList ? kOpGatherLogit : kOpRangeLogit;
        state = sm.hit_cnt <= kSmpList ? kAfterGather : kAfterRange;
        return;
      case kAfterRange:
        c.klo = 0xFFFFFFFFu;
        c.khi = 0;
        for (int r = 0; r < cs; ++r) {
          c.klo = min(c.klo, sm.xlo[r]);
          c.khi = max(c.khi, sm.xhi[r]);
        }
        refine = true;
        break;
      case kAfterKeyHist: {
        locate();
        c.khi -= static_cast<uint32_t>(sm.hit) << c.shift;
        const uint32_t width = (1u << c.shift) - 1u;
        if (c.khi - c.klo > width) c.klo = c.khi - width;
        refine = true;
        break;
      }
      case kAfterCount: {
        uint64_t a = tid < cs * kSmpWarps ? sm.xcnt[tid] : 0, b = 0;
        const uint64_t mine = a;
        block_scan(a, b);
        const uint64_t need = sm.need;
        if (a - mine < need && need <= a) {
          sm.hit = tid;
          sm.hit_cnt = static_cast<uint32_t>(need - 1 - (a - mine));
        }
        __syncthreads();
        c.op = kOpFindEqual;
        c.rank = sm.hit / kSmpWarps;
        c.warp = sm.hit % kSmpWarps;
        c.nth = static_cast<int>(sm.hit_cnt);
        state = kAfterFind;
        return;
      }
      case kAfterFind:
        if (tid == 0) {
          sm.cut_key = c.khi;
          sm.cut_index = static_cast<int>(sm.found);
        }
        found = true;
        break;
      case kAfterGather: {
        const int n = collect();
        // how many of them are needed
        const int at =
            sm.by_mass ? 1 + __syncthreads_count(tid < n && sm.acc_mass + sm.run[tid] < sm.target)
                       : static_cast<int>(sm.target - sm.acc_cnt);
        if (tid == 0) {
          const uint64_t key = sm.sorted[at - 1];
          sm.cut_key = static_cast<uint32_t>(key >> 32);
          sm.cut_index = static_cast<int>(~static_cast<uint32_t>(key));
          sm.mass = sm.acc_mass + sm.run[at - 1];
        }
        found = true;
        break;
      }
      default:   // kAfterSum
        pick(c);
        return;
    }
    if (refine) {
      const uint32_t span = c.khi - c.klo;
      if (sm.hit_cnt <= kSmpList) {
        c.op = kOpGatherKey;
        state = kAfterGather;
        return;
      }
      if (span > 0) {
        c.shift = max(0, 32 - __clz(span) - 10);
        c.op = kOpHistKey;
        state = kAfterKeyHist;
        return;
      }
      // equal keys: the first `need` of them in index order
      const uint64_t w = weight(smp_value(c.khi));
      const uint64_t need = sm.by_mass ? (sm.target - sm.acc_mass + w - 1) / w
                                       : sm.target - sm.acc_cnt;
      __syncthreads();
      if (tid == 0) {
        sm.need = need;
        sm.mass = sm.acc_mass + need * w;
        sm.cut_key = c.khi;
        sm.cut_index = INT_MAX;
      }
      if (need < sm.hit_cnt) {
        c.op = kOpCountEqual;
        state = kAfterCount;
        return;
      }
      found = true;
    }
    if (found) {
      const bool more = by_p && !sm.by_mass;
      __syncthreads();
      if (more) {
        search(c, true, share(sm.mass));
        return;
      }
      c.op = kOpSum;
      c.khi = sm.cut_key;
      c.nth = sm.cut_index;
      state = kAfterSum;
    }
  };

  SmpCmd c = {};
  while (true) {
    if (rank == 0) {
      decide(c);
      __syncthreads();
      if (tid < cs) *smp_remote(&sm.cmd, tid) = c;
    }
    smp_cluster_sync();
    c = sm.cmd;
    if (c.op == kOpDone) return;
    carry_out(c);
    if (c.op == kOpPick) return;
    smp_cluster_sync();
  }
}

// Rows are cut so that two CTAs fit an SM (one's passes run while the other's
// row arrives); few rows over as many CTAs as leave each some thousand tokens
// (a cluster of more than eight lies in one GPC, so only for a handful of rows).
constexpr int kSmpSliceBytes = 80 * 1024;
constexpr int kSmpMostBytes = 176 * 1024;   // one CTA an SM

template <typename T>
dfv_status sample_launch(SampleParams p, cudaStream_t stream) {
  constexpr int kV = SmpVec<T>::kN;
  const int64_t vecs = p.vocab / kV + 2;
  const int most = p.n_rows <= 4 ? 16 : p.n_rows <= 37 ? 8 : p.n_rows <= 75 ? 4 : 1;
  int cs = 1;
  auto slice = [&]() { return (vecs + cs - 1) / cs + 2; };   // head and tail vectors beside
  while (cs < kSmpMaxCluster &&
         (slice() * 16 > kSmpSliceBytes || (cs < most && p.vocab > cs * 8192)))
    cs <<= 1;
  if (slice() * 16 > kSmpMostBytes) return DFV_ERR_UNSUPPORTED;
  p.slice_vecs = static_cast<int>(slice());
  const int smem = static_cast<int>((sizeof(SmpSmem) + 127) / 128 * 128) + p.slice_vecs * 16;
  static std::atomic<int> allowed[64];   // per device
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return DFV_ERR_CUDA;
  if (!allowed[dev].load(std::memory_order_acquire)) {
    constexpr int kMost = static_cast<int>((sizeof(SmpSmem) + 127) / 128 * 128) + kSmpMostBytes;
    if (cudaFuncSetAttribute(sample_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kMost) != cudaSuccess ||
        cudaFuncSetAttribute(sample_kernel<T>, cudaFuncAttributeNonPortableClusterSizeAllowed,
                             1) != cudaSuccess)
      return DFV_ERR_CUDA;
    allowed[dev].store(1, std::memory_order_release);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.n_rows) * cs);
  cfg.blockDim = dim3(kSmpThreads);
  cfg.dynamicSmemBytes = smem;
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
  return cudaLaunchKernelEx(&cfg, sample_kernel<T>, p) == cudaSuccess ? DFV_OK : DFV_ERR_CUDA;
}

// What both entry points check; true: `st` is the answer.
bool sample_refused(int n_rows, int vocab, int dtype, const void* logits, int64_t stride_row,
                    const float* uniform, const dfv_sampling* s, const int32_t* token,
                    const float* logprob, dfv_status& st) {
  st = DFV_ERR_UNSUPPORTED;
  if (dtype != DFV_DTYPE_F32 && dtype != DFV_DTYPE_BF16) return true;
  if (vocab > kSmpMaxVocab) return true;
  st = DFV_ERR_INVALID;
  const size_t size = dtype == DFV_DTYPE_F32 ? 4 : 2;
  if (n_rows < 0 || n_rows > (1 << 26) || vocab < 1 || !s || (n_rows > 1 && stride_row < vocab))
    return true;
  if (n_rows == 0) {
    st = DFV_OK;
    return true;
  }
  return !logits || !uniform || !token || !aligned(logits, size) || !aligned(uniform, 4) ||
         !aligned(token, 4) || !aligned(logprob, 4) || !aligned(s->temperature, 4) ||
         !aligned(s->top_k, 4) || !aligned(s->top_p, 4) || !aligned(s->min_p, 4);
}

dfv_status sample_any(const SampleParams& p, int dtype, cudaStream_t stream) {
  return dtype == DFV_DTYPE_F32 ? sample_launch<float>(p, stream)
                                : sample_launch<__nv_bfloat16>(p, stream);
}

}  // namespace dfv

extern "C" dfv_status dfv_sample(int n_rows, int vocab, int logits_dtype, const void* logits,
                                 int64_t stride_row, const float* uniform,
                                 const dfv_sampling* sampling, int32_t* token, float* logprob,
                                 uint32_t* status, dfv_stream_t stream) {
  using namespace dfv;
  dfv_status st;
  if (sample_refused(n_rows, vocab, logits_dtype, logits, stride_row, uniform, sampling, token,
                     logprob, st))
    return st;
  SampleParams p = {};
  p.n_rows = n_rows;
  p.vocab = vocab;
  p.logits = logits;
  p.stride = stride_row;
  p.uniform = uniform;
  p.s = *sampling;
  p.token = token;
  p.logprob = logprob;
  p.status = status;
  return sample_any(p, logits_dtype, static_cast<cudaStream_t>(stream));
}

extern "C" size_t dfv_sample_accept_workspace_bytes(int n_nodes, int vocab) {
  return n_nodes < 1 || n_nodes > dfv::kMaxNodes || vocab < 1 || vocab > dfv::kSmpMaxVocab ? 0
                                                                                          : 256;
}

extern "C" dfv_status dfv_sample_accept(int n_nodes, int vocab, int logits_dtype,
                                        const void* logits, int64_t stride_row,
                                        const float* uniform, const dfv_sampling* sampling,
                                        const int32_t* parent, const int32_t* tokens,
                                        int32_t* target, float* logprob, int32_t* accept_len,
                                        int32_t* path, int32_t* out_tokens, void* workspace,
                                        size_t workspace_bytes, uint32_t* status,
                                        dfv_stream_t stream) {
  using namespace dfv;
  if (n_nodes < 1 || n_nodes > kMaxNodes) return DFV_ERR_INVALID;
  dfv_status st;
  if (sample_refused(n_nodes, vocab, logits_dtype, logits, stride_row, uniform, sampling, target,
                     logprob, st))
    return st;
  if (!parent || !tokens || !accept_len || !path || !out_tokens || !workspace ||
      !aligned(parent, 4) || !aligned(tokens, 4) || !aligned(accept_len, 4) ||
      !aligned(path, 4) || !aligned(out_tokens, 4) || !aligned(workspace, 256))
    return DFV_ERR_INVALID;
  if (workspace_bytes < dfv_sample_accept_workspace_bytes(n_nodes, vocab))
    return DFV_ERR_WORKSPACE;
  SampleParams p = {};
  p.n_rows = n_nodes;
  p.vocab = vocab;
  p.logits = logits;
  p.stride = stride_row;
  p.uniform = uniform;
  p.s = *sampling;
  p.token = target;
  p.logprob = logprob;
  p.status = status;
  p.parent = parent;
  p.tokens = tokens;
  p.accept_len = accept_len;
  p.path = path;
  p.out_tokens = out_tokens;
  p.ticket = static_cast<unsigned int*>(workspace);
  return sample_any(p, logits_dtype, static_cast<cudaStream_t>(stream));
}
