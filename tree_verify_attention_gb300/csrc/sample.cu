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
// 2^(j/32) in 32 bits and a quartic for the rest, t = (x - base) log2(e) / T in
// two floats: off by up to 2^-29 of the weight, which many weights average out.
// The few largest do not, so about the 24 largest tokens are weighed in 64 bits
// throughout. Sums of integers have no order, so every pass over the row agrees
// with every other and nothing depends on how the row is split.
//
// A row belongs to a cluster of 1 to 16 CTAs that keep it in shared memory:
// it is read from memory once, and passes over it run at shared memory's rate.
// The first CTA decides, the others carry out what it asks for. Passes:
//
//   1. maximum, while the row arrives, and the maxima of groups of tokens, about
//      twice as many as top-k says (up to 256; 24 without it): the k-th largest
//      of these is reached by k tokens at least, and by not many more;
//   2. top-k of up to 256: the tokens that reach that bound, into a list. Else
//      the sum of all weights, a list of the tokens within 2^-12 of the largest,
//      and counts of every eighth piece of the row by bins of the logit.
//      A list that holds both cuts (a model that is reasonably sure) is sorted
//      in the first CTA, and the token comes from it;
//   3. otherwise the counts give a window for the cut, mostly from below: what
//      top-p cuts off has a known weight in many light tokens, whose sampled
//      counts are far surer than those of the few heavy ones (1024 rows of
//      151936, top-p 0.99: 924 us, from above alone 1560). The tokens above the
//      window are weighed, the ones in it gathered in index order, and what
//      follows runs over these alone (over the whole row where they are too many
//      or the cut lies elsewhere): counts and weights by bins of the logit, the
//      bin with the cut, its tokens sorted (a bin of more than 512 is cut by its
//      keys' bits; equal keys are counted in index order);
//   4. the sum of the kept weights per warp, and the warp with the token once
//      more.
//
// Without top-k and top-p pass 2 is pass 4. The kernel is bound by the integer
// work on weights (about 30 cycles of a scheduler for 32 lanes, in passes 2 and 3)
// and, for few rows, by the chain of decisions in the first CTA. 1024 rows of
// 151936 bf16 logits, a few of which stand out: greedy 115 us, no cut 297, top-k 50
// 223, top-p 0.9 at 0.7 303, top-p 0.95 779; 23 rows 7, 19, 14, 20, 45; one f32 row
// 6, 14, 14, 15, 34. (Normal logits of deviation 2 alone have flatter cuts: top-p
// 0.95 1091, 23 rows 57.)

#include <atomic>
#include <climits>

#include "common.cuh"
#include "tc.cuh"

namespace dfv {

constexpr int kSmpThreads = 512;
constexpr int kSmpWarps = kSmpThreads / 32;
constexpr int kSmpBins = kSmpThreads;
constexpr int kSmpBinBits = 9;
constexpr int kSmpList = kSmpThreads;      // one sorted token a thread
constexpr int kSmpTopMost = 256;           // top-k by group maxima
constexpr int kSmpHeavy = 24;              // tokens weighed in 64 bits, about
constexpr int kSmpGroups = 1024;           // of them, at most
constexpr int kSmpGathered = 384;          // of a warp
constexpr int kSmpSample = 8;              // turns of a warp for one whose tokens are counted
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
};

// round(2^(63 + j / 32))
__constant__ uint64_t kSmpExp2[32] = {
    0x8000000000000000ull, 0x82CD8698AC2BA1D7ull, 0x85AAC367CC487B15ull, 0x88980E8092DA8527ull,
    0x8B95C1E3EA8BD6E7ull, 0x8EA4398B45CD53C0ull, 0x91C3D373AB11C336ull, 0x94F4EFA8FEF70961ull,
    0x9837F0518DB8A96Full, 0x9B8D39B9D54E5539ull, 0x9EF5326091A111AEull, 0xA27043030C496819ull,
    0xA5FED6A9B15138EAull, 0xA9A15AB4EA7C0EF8ull, 0xAD583EEA42A14AC6ull, 0xB123F581D2AC2590ull,
    0xB504F333F9DE6484ull, 0xB8FBAF4762FB9EE9ull, 0xBD08A39F580C36BFull, 0xC12C4CCA66709456ull,
    0xC5672A115506DADDull, 0xC9B9BD866E2F27A3ull, 0xCE248C151F8480E4ull, 0xD2A81D91F12AE45Aull,
    0xD744FCCAD69D6AF4ull, 0xDBFBB797DAF23755ull, 0xE0CCDEEC2A94E111ull, 0xE5B906E77C8348A8ull,
    0xEAC0C6E7DD24392Full, 0xEFE4B99BDCDAF5CBull, 0xF5257D152486CC2Cull, 0xFA83B2DB722A033Aull,
};

template <bool kOn> struct SmpFlag {
  static constexpr bool value = kOn;
};

enum SmpState {
  kStart, kAfterHist, kAfterRange, kAfterKeyHist, kAfterCount, kAfterFind, kAfterGather, kAfterSum
};

enum SmpOp {
  kOpDone, kOpCompact, kOpHistLogit, kOpGatherLogit, kOpRangeLogit, kOpHistKey, kOpGatherKey,
  kOpCountEqual, kOpFindEqual, kOpSum, kOpPick
};

struct SmpCmd {
  int op, bin, shift, rank, warp, nth;
  int gathered;          // over the gathered tokens
  int under_list;        // the window ends where the list begins
  float from, upto;      // gather the tokens of logits in [from, upto)
  float bin0, bins;      // bin of a logit v: (bin0 - v) bins
  uint32_t khi, klo;     // keys, both included
  uint64_t target, total;
};

struct SmpSmem {
  uint32_t cnt[kSmpBins], mlo[kSmpBins], mhi[kSmpBins];   // a bin's count and weight
  alignas(16) uint64_t buf[kSmpList];   // this CTA's list; first CTA: then the cluster's,
                                        // then its weights in order
  union {
    uint64_t sorted[kSmpList];   // in order
    alignas(16) float gmax[kSmpGroups];      // before: the cluster's group maxima
  };
  uint64_t run[kSmpList];      // running weights
  uint32_t sampled[kSmpBins];  // counts of every eighth piece
  uint16_t gathered[kSmpWarps][kSmpGathered];   // places in the slice, ascending
  uint32_t table[32];          // 2^(31 + j / 32): an entry a bank
  float ftable[32];            // 2^(j / 32)
  uint64_t wtot[2][kSmpWarps];
  float wmax[kSmpWarps];
  float xmax[kSmpMaxCluster];
  // first CTA: what the others report
  uint64_t xsum[kSmpMaxCluster * kSmpWarps], xlmass[kSmpMaxCluster * kSmpWarps];
  uint32_t xcnt[kSmpMaxCluster * kSmpWarps];
  int xlist[kSmpMaxCluster];
  uint32_t xlo[kSmpMaxCluster], xhi[kSmpMaxCluster];
  uint32_t found, over;        // a place; warps whose gathered tokens did not fit
  // parameters of the row
  float t_inv_hi, t_inv_lo, temperature, top_p, u, ln_hi, ln_lo;
  int top_k, bad;
  int list_n;
  float bound;
  uint32_t lo, hi;
  SmpCmd cmd;
  // first CTA: a search, its hit, and the cut so far with the weight up to it
  bool by_mass;
  int hit, hit2, list_all;
  uint32_t hit_cnt;
  uint64_t target, acc_cnt, acc_mass, need, mass, binned;
  uint64_t mass_all;     // of all tokens
  float sigma2[2];       // variance of the cut's estimate from above, from below
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
  static __device__ __forceinline__ float2 pair(const void* x, int i) {
    return static_cast<const float2*>(x)[i];
  }
};
template <> struct SmpVec<__nv_bfloat16> {
  static constexpr int kN = 8;
  static __device__ __forceinline__ float at(const uint4& v, int i) {
    const uint32_t w = i < 2 ? v.x : i < 4 ? v.y : i < 6 ? v.z : v.w;
    return __uint_as_float(i & 1 ? w & 0xFFFF0000u : w << 16);
  }
  static __device__ __forceinline__ __nv_bfloat16 low() { return __float2bfloat16(-INFINITY); }
  static __device__ __forceinline__ float2 pair(const void* x, int i) {
    const uint32_t w = static_cast<const uint32_t*>(x)[i];
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  }
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

// Two float32 operations in one instruction.
__device__ __forceinline__ float2 smp_add2(float2 a, float2 b) {
  add2(a.x, a.y, a.x, a.y, b.x, b.y);
  return a;
}
__device__ __forceinline__ float2 smp_fma2(float2 a, float2 b, float2 c) {
  fma2(c.x, c.y, a.x, a.y, b.x, b.y, c.x, c.y);
  return c;
}
__device__ __forceinline__ float2 smp_both(float x) { return make_float2(x, x); }

// 2^(k / 32 + f + g) in 64 bits, |f + g| <= 2^-6, in the units that `s` gives the
// other weights. The series of 2^r - 1 by
// Horner's rule in 64-bit fractions, up to r^6 (the next term is below 2^-54).
__device__ __noinline__ uint64_t smp_heavy_weight(float f, float g, int k, uint32_t s) {
  const int64_t r = __float2ll_rn(f * 0x1p60f) + __float2ll_rn(g * 0x1p60f);
  const bool neg = r < 0;
  const uint64_t a = __umul64hi(static_cast<uint64_t>(neg ? -r : r) << 3,
                                0xB17217F7D1CF79ACull);   // |r| ln2, times 2^63
  // 1 + z + z^2 / 2! ..., z = +-a: sums of magnitudes by sign, times 2^63
  uint64_t even = 0, odd = a, power = a;
#pragma unroll
  for (int i = 2; i <= 6; ++i) {
    power = (__umul64hi(power, a) << 1) / static_cast<uint64_t>(i);
    if (i & 1) odd += power;
    else even += power;
  }
  const uint64_t one = 1ull << 63;
  const uint64_t e = neg ? one + even - odd : one + even + odd;   // e^z, below 2^64
  const uint64_t t = kSmpExp2[k & 31];                            // below 2^64
  const uint64_t w = __umul64hi(t, e);                            // 2^(62 + t's fraction)
  return s > 64 ? 0 : w >> (s - 1);
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
  if (__shfl_sync(0xFFFFFFFFu, last, 0)) {
    __syncwarp();   // what lane 0 has acquired is every lane's (a shuffle orders no memory)
    smp_walk(p, lane);
  }
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
  if (tid < 32) {
    const uint64_t t = kSmpExp2[tid];
    sm.table[tid] = static_cast<uint32_t>((t + 0x80000000ull) >> 32);
    sm.ftable[tid] = static_cast<float>(t) * 0x1p-63f;
  }
  sm.sampled[tid] = 0;
  if (tid == 0) sm.list_n = sm.over = 0;
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
    // log2(e) / temperature in two floats
    const float hi = 1.44269502f / temp;
    sm.t_inv_hi = hi;
    sm.t_inv_lo = (fmaf(-hi, temp, 1.44269502f) + 1.92596303e-8f) / temp;
    sm.temperature = temp;
    sm.top_p = top_p;
    sm.u = u;
    sm.top_k = p.s.top_k ? p.s.top_k[row] : p.s.top_k_all;
    // ln(max(min(min_p, 1), 2^-40)) in two (64 bits only where it is used: an
    // operation takes 76 cycles)
    const double ln = min_p > 0x1p-40f ? log(static_cast<double>(fminf(min_p, 1.0f)))
                                       : -27.725887222397812377;
    sm.ln_hi = static_cast<float>(ln);
    sm.ln_lo = static_cast<float>(ln - static_cast<double>(sm.ln_hi));
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
  const bool by_k = sm.top_k > 0 && sm.top_k < p.vocab, by_p = sm.top_p < 1.0f;
  // groups of neighbouring threads, about twice as many in the cluster as the
  // bound that is asked of them
  const bool by_groups = by_k && sm.top_k <= kSmpTopMost;
  const int want = by_groups ? sm.top_k : kSmpHeavy;
  int lanes = 32;   // of a group
  while (lanes > 1 && cs * (kSmpThreads / lanes) < 2 * want) lanes >>= 1;
  const int groups = kSmpThreads / lanes;   // of a CTA
  float gm = mx;
  for (int o = lanes >> 1; o > 0; o >>= 1) gm = fmaxf(gm, __shfl_xor_sync(0xFFFFFFFFu, gm, o));
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
  if (tid % lanes == 0) {
    for (int r = 0; r < cs; ++r) *smp_remote(&sm.gmax[rank * groups + tid / lanes], r) = gm;
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
  // Passes go by pairs of tokens, a pair a lane: their code is short, which
  // counts for more than wide loads (what runs a few times a row comes from the
  // instruction cache's far end). A warp's pairs are neighbours, so that warps
  // are in index order.
  const int n_pairs = n_vecs * (kV / 2);
  const int per = (n_pairs + kSmpWarps - 1) / kSmpWarps;
  const int u0 = min(n_pairs, warp * per), u1 = min(n_pairs, u0 + per);
  if (sm.temperature < kSmpMinT) {
    uint32_t best = 0xFFFFFFFFu;
    for (int u = u0 + lane; u < u1 && best == 0xFFFFFFFFu; u += 32) {
      const float2 v = SmpVec<T>::pair(xs, u);
      if (v.x == m || v.y == m) best = static_cast<uint32_t>(first + 2 * u + (v.x == m ? 0 : 1));
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

  // ---- the bound that `want` tokens reach at least, the same in every CTA
  {
    const int all = cs * groups;
    for (int i = tid; i < all; i += kSmpThreads) {
      const float g = sm.gmax[i];
      int above = 0, same = 0;
#pragma unroll 4
      for (int j = 0; j < all; j += 4) {   // (at least 16 groups, a power of two)
        const float4 o = *reinterpret_cast<const float4*>(&sm.gmax[j]);
        above += (o.x > g) + (o.y > g) + (o.z > g) + (o.w > g);
        same += (o.x >= g) + (o.y >= g) + (o.z >= g) + (o.w >= g);
      }
      if (above < want && same >= want) sm.bound = g;   // the same value from each such thread
    }
    __syncthreads();
  }
  const float heavy = fmaxf(sm.bound, -3.4028235e38f);

  // ---- weights. |m| / T up to 2^12: t = x / T log2(e) itself, to 2^-36; above,
  // tokens that count lie so near the maximum that x - m is exact.
  const float chi = sm.t_inv_hi, clo = sm.t_inv_lo, temp = sm.temperature;
  const float base = fabsf(m) * chi <= 4096.0f ? 0.0f : m;
  constexpr float kMagic = 12582912.0f;   // 1.5 * 2^23: the sum's low bits are the integer
  // t = d log2(e) / T = k / 32 + f + g with k an integer (in the low bits of
  // `k`) and |f| <= 2^-6, of two values at a time
  auto split = [&](float2 v, float2& k, float2& g) {
    const float2 d = smp_add2(v, smp_both(-base)), c = smp_both(chi);
    const float2 th = smp_fma2(d, c, smp_both(-0.0f));
    g = smp_fma2(d, smp_both(clo), smp_fma2(d, c, make_float2(-th.x, -th.y)));
    k = smp_fma2(th, smp_both(32.0f), smp_both(kMagic));
    return smp_fma2(smp_add2(k, smp_both(-kMagic)), smp_both(-0.03125f), th);
  };
  // s of the maximum is 20: the largest weight is in [2^43, 2^44]
  int top;
  {
    float2 k, g;
    split(smp_both(m), k, g);
    top = 20 + (__float_as_int(k.x) >> 5);
  }
  // Weights of two values, zero where `on` is not set; the largest tokens' are
  // put right if `heavies` says so.
  auto weights_of = [&](float2 v, bool on0, bool on1, uint64_t& w0, uint64_t& w1, auto heavies) {
    float2 k, g;
    const float2 f = split(v, k, g), r = smp_add2(f, g);
    // 2^31 (2^r - 1), |r| <= 2^-6: ln2^i / i!; the next term is below 2^-39
    float2 q = smp_fma2(r, smp_both(0.0096181291f * 0x1p31f), smp_both(0.055504109f * 0x1p31f));
    q = smp_fma2(r, q, smp_both(0.24022651f * 0x1p31f));
    q = smp_fma2(r, q, smp_both(0.69314718f * 0x1p31f));
    q = smp_fma2(r, q, smp_both(0.0f));
    const int k0 = __float_as_int(k.x), k1 = __float_as_int(k.y);
    uint32_t f0 = sm.table[k0 & 31] +
                  static_cast<uint32_t>(__float2int_rn(sm.ftable[k0 & 31] * q.x));
    uint32_t f1 = sm.table[k1 & 31] +
                  static_cast<uint32_t>(__float2int_rn(sm.ftable[k1 & 31] * q.y));
    f0 = on0 ? f0 : 0u;
    f1 = on1 ? f1 : 0u;
    // f 2^(32 - s), s at least 20 (PTX shifts stop at the width, C's may not)
    const uint32_t s0 = top - (k0 >> 5), s1 = top - (k1 >> 5);
    asm("{\n\t.reg .b64 a;\n\tmov.b64 a, {0, %1};\n\tshr.u64 %0, a, %2;\n\t}"
        : "=l"(w0) : "r"(f0), "r"(s0));
    asm("{\n\t.reg .b64 a;\n\tmov.b64 a, {0, %1};\n\tshr.u64 %0, a, %2;\n\t}"
        : "=l"(w1) : "r"(f1), "r"(s1));
    if (decltype(heavies)::value && fmaxf(v.x, v.y) >= heavy) {
      if (on0 && v.x >= heavy) w0 = smp_heavy_weight(f.x, g.x, k0, s0);
      if (on1 && v.y >= heavy) w1 = smp_heavy_weight(f.y, g.y, k1, s1);
    }
  };
  auto weight2 = [&](float2 v, bool on0, bool on1, uint64_t& w0, uint64_t& w1) {
    weights_of(v, on0, on1, w0, w1, SmpFlag<true>());
  };
  auto weight = [&](float v) {
    uint64_t w0, w1;
    weight2(smp_both(v), true, false, w0, w1);
    return w0;
  };
  // below: no weight left of 2^-44; within 2^-12 of the largest; kept by min-p
  // (finite, so that -inf is below all three)
  const float tau_w = fmaxf(m - 43.0f * 0.69314718f * temp, -3.4028235e38f);
  float tau_l = fmaxf(m - 12.0f * 0.69314718f * temp, -3.4028235e38f);
  float tau_0;   // the smallest float at or above m + T ln(min-p)
  {
    const float a = temp * sm.ln_hi, ae = fmaf(temp, sm.ln_hi, -a) + temp * sm.ln_lo;
    const float b = m + a, bb = b - m;
    const float be = ((m - (b - bb)) + (a - bb)) + ae;
    tau_0 = fmaxf(be > 0.0f ? nextafterf(b, INFINITY) : b, -3.4028235e38f);
  }
  const float bin_scale = (kSmpBins - 0.5f) / (43.0f * 0.69314718f) / temp;
  auto logit_bin = [&](float v) {   // monotone: each operation is
    return min(static_cast<int>((m - v) * bin_scale), kSmpBins - 1);
  };
  // of a search: the window's logits, or all, over all bins (a window of equal
  // logits has one: 0 times infinity converts to 0)
  auto command_bin = [](const SmpCmd& c, float v) {
    return min(static_cast<int>((c.bin0 - v) * c.bins), kSmpBins - 1);
  };

  // f(logits, row index of the first, which of the two) over this warp's tokens:
  // the gathered ones, one a lane, or all, a pair a lane.
  int n_gathered = 0;
  uint64_t above = 0, listed = 0;   // a lane's weight above them, and in the list
  auto each = [&](const SmpCmd& c, auto f) {
    const int n = c.gathered ? n_gathered : u1 - u0;
#pragma unroll 1
    for (int i = lane; i < n; i += 32) {
      if (c.gathered) {
        const int at = sm.gathered[warp][i];
        f(make_float2(static_cast<float>(xe[at]), -INFINITY), first + at, false);
      } else {
        f(SmpVec<T>::pair(xs, u0 + i), first + 2 * (u0 + i), true);
      }
    }
  };
  auto key_of = [&](float v, int i) {
    return (static_cast<uint64_t>(smp_order(v)) << 32) | static_cast<uint32_t>(~i);
  };
  auto push = [&](float v, int i) {
    const int k = atomicAdd(&sm.list_n, 1);
    if (k < kSmpList) sm.buf[k] = key_of(v, i);
  };
  auto tell_sum = [&](uint64_t s, uint64_t* where) {
    s = smp_warp_sum(s);
    if (lane == 0) *smp_remote(&where[rank * kSmpWarps + warp], 0) = s;
  };

  // ---- pass 2
  if (by_groups) {
    tau_l = heavy;
#pragma unroll 1
    for (int u = u0 + lane; u < u1; u += 32) {
      const float2 x = SmpVec<T>::pair(xs, u);
      if (fmaxf(x.x, x.y) >= tau_l) {
        if (x.x >= tau_l) push(x.x, first + 2 * u);
        if (x.y >= tau_l) push(x.y, first + 2 * u + 1);
      }
    }
  } else {
    uint64_t s = 0;
    const bool filter = by_k || by_p;
    const float from = filter ? tau_w : tau_0;
    // the largest and the listed tokens are few: one test for two pairs
    const float rare = filter ? fminf(heavy, tau_l) : heavy;
    auto fix = [&](float2 x, int u, uint64_t& w0, uint64_t& w1) {
      if (!(fmaxf(x.x, x.y) >= rare)) return;
      weight2(x, x.x >= from, x.y >= from, w0, w1);
      if (filter && x.x >= tau_l) {
        push(x.x, first + 2 * u);
        listed += w0;
      }
      if (filter && x.y >= tau_l) {
        push(x.y, first + 2 * u + 1);
        listed += w1;
      }
    };
    int turn = 0;
#pragma unroll 1
    for (int u = u0 + lane; u < u1; u += 64, turn += 2) {
      const bool two = u + 32 < u1;
      const float2 x = SmpVec<T>::pair(xs, u);
      const float2 y = two ? SmpVec<T>::pair(xs, u + 32) : smp_both(-INFINITY);
      uint64_t w0, w1, w2, w3;
      weights_of(x, x.x >= from, x.y >= from, w0, w1, SmpFlag<false>());
      weights_of(y, y.x >= from, y.y >= from, w2, w3, SmpFlag<false>());
      if (fmaxf(fmaxf(x.x, x.y), fmaxf(y.x, y.y)) >= rare) {
        fix(x, u, w0, w1);
        fix(y, u + 32, w2, w3);
      }
      s += (w0 + w1) + (w2 + w3);
      if (filter && turn % kSmpSample == 0) {
        if (x.x >= tau_w) atomicAdd(&sm.sampled[logit_bin(x.x)], 1u);
        if (x.y >= tau_w) atomicAdd(&sm.sampled[logit_bin(x.y)], 1u);
      }
    }
    tell_sum(s, sm.xsum);
    if (filter) tell_sum(listed, sm.xlmass);
  }
  if (by_k || by_p) {
    __syncthreads();
    if (tid == 0) *smp_remote(&sm.xlist[rank], 0) = sm.list_n;
  }
  smp_cluster_sync();

  auto hist_add = [&](int b, uint64_t w) {
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
      case kOpCompact: {
        // the window's tokens in index order, and the count and weight of those
        // above it
        n_gathered = 0;
        above = c.under_list ? listed : 0;
        uint32_t n_above = 0;
#pragma unroll 1
        for (int u = u0; u < u1; u += 32) {
          const bool on = u + lane < u1;
          // (behind the run: neither in the window nor above it, whatever its bounds)
          const float2 x = on ? SmpVec<T>::pair(xs, u + lane) : smp_both(NAN);
          const bool over0 = x.x >= c.upto, over1 = x.y >= c.upto;
          const bool in0 = x.x >= c.from && !over0, in1 = x.y >= c.from && !over1;
          if (!c.under_list && (over0 || over1)) {
            uint64_t w0, w1;
            weight2(x, over0, over1, w0, w1);
            above += w0 + w1;
            n_above += (over0 ? 1 : 0) + (over1 ? 1 : 0);
          }
          const unsigned b0 = __ballot_sync(0xFFFFFFFFu, in0), b1 = __ballot_sync(0xFFFFFFFFu, in1);
          if (b0 | b1) {
            const unsigned below = (1u << lane) - 1u;
            int at = n_gathered + __popc(b0 & below) + __popc(b1 & below);
            if (in0 && at < kSmpGathered)
              sm.gathered[warp][at] = static_cast<uint16_t>(2 * (u + lane));
            at += in0 ? 1 : 0;
            if (in1 && at < kSmpGathered)
              sm.gathered[warp][at] = static_cast<uint16_t>(2 * (u + lane) + 1);
            n_gathered += __popc(b0) + __popc(b1);
          }
        }
        n_above = __reduce_add_sync(0xFFFFFFFFu, n_above);
        if (lane == 0) *smp_remote(&sm.xcnt[rank * kSmpWarps + warp], 0) = n_above;
        tell_sum(above, sm.xsum);
        if (n_gathered > kSmpGathered) {
          n_gathered = 0;
          if (lane == 0) atomicAdd(smp_remote(&sm.over, 0), 1u);
        }
        __syncwarp();
      }
        [[fallthrough]];
      case kOpHistLogit:
      case kOpHistKey:
        sm.cnt[tid] = sm.mlo[tid] = sm.mhi[tid] = 0;
        __syncthreads();
        each(c, [&](float2 v, int, bool) {
          bool in0, in1;
          int b0, b1;
          if (c.op != kOpHistKey) {
            in0 = v.x >= tau_w;
            in1 = v.y >= tau_w;
            b0 = command_bin(c, v.x);
            b1 = command_bin(c, v.y);
          } else {
            const uint32_t o0 = smp_order(v.x), o1 = smp_order(v.y);
            in0 = o0 <= c.khi && o0 >= c.klo;
            in1 = o1 <= c.khi && o1 >= c.klo;
            b0 = (c.khi - o0) >> c.shift;
            b1 = (c.khi - o1) >> c.shift;
          }
          if (!in0 && !in1) return;
          uint64_t w0, w1;
          weight2(v, in0, in1, w0, w1);
          if (in0) hist_add(b0, w0);
          if (in1) hist_add(b1, w1);
        });
        break;
      case kOpGatherLogit:
      case kOpGatherKey:
        if (tid == 0) sm.list_n = 0;
        __syncthreads();
        each(c, [&](float2 v, int i, bool) {
          auto in = [&](float z) {
            if (c.op == kOpGatherLogit) return z >= tau_w && command_bin(c, z) == c.bin;
            const uint32_t o = smp_order(z);
            return o <= c.khi && o >= c.klo;
          };
          if (in(v.x)) push(v.x, i);
          if (in(v.y)) push(v.y, i + 1);
        });
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
        each(c, [&](float2 v, int, bool) {
          auto add = [&](float z) {
            if (z >= tau_w && command_bin(c, z) == c.bin) {
              lo = min(lo, smp_order(z));
              hi = max(hi, smp_order(z));
            }
          };
          add(v.x);
          add(v.y);
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
        each(c, [&](float2 v, int, bool) {
          n += (smp_order(v.x) == c.khi) + (smp_order(v.y) == c.khi);
        });
        n = __reduce_add_sync(0xFFFFFFFFu, n);
        if (lane == 0) *smp_remote(&sm.xcnt[rank * kSmpWarps + warp], 0) = n;
        break;
      }
      case kOpFindEqual:   // the nth of a warp's equal keys
        if (rank == c.rank && warp == c.warp) {
          int before = 0;
          const int n = c.gathered ? n_gathered : (u1 - u0) * 2;
          for (int i = 0; i < n; i += 32) {
            int at = 0;
            if (i + lane < n) at = c.gathered ? sm.gathered[warp][i + lane] : u0 * 2 + i + lane;
            const unsigned same = __ballot_sync(
                0xFFFFFFFFu, i + lane < n && smp_order(static_cast<float>(xe[at])) == c.khi);
            if ((same >> lane) & 1u && before + __popc(same & ((1u << lane) - 1u)) == c.nth)
              *smp_remote(&sm.found, 0) = static_cast<uint32_t>(first + at);
            before += __popc(same);
          }
        }
        break;
      case kOpSum: {
        uint64_t s = c.gathered ? above : 0;
        each(c, [&](float2 v, int i, bool both) {
          const bool k0 = kept(c, v.x, i), k1 = both && kept(c, v.y, i + 1);
          if (!k0 && !k1) return;
          uint64_t w0, w1;
          weight2(v, k0, k1, w0, w1);
          s += w0 + w1;
        });
        tell_sum(s, sm.xsum);
        break;
      }
      case kOpPick:
        // the token at which the running sum exceeds the target, in the run of
        // one warp: all warps of its CTA take a sixteenth of it each
        if (rank == c.rank) {
          const int r0 = min(n_pairs, c.warp * per), r1 = min(n_pairs, r0 + per);
          const int part = (r1 - r0 + kSmpWarps - 1) / kSmpWarps;
          const int q0 = min(r1, r0 + warp * part), q1 = min(r1, q0 + part);
          auto pair_weights = [&](int u, uint64_t& w0, uint64_t& w1) {
            w0 = w1 = 0;
            if (u >= q1) return;
            const float2 x = SmpVec<T>::pair(xs, u);
            weight2(x, kept(c, x.x, first + 2 * u), kept(c, x.y, first + 2 * u + 1), w0, w1);
          };
          uint64_t s = 0, w0, w1;
#pragma unroll 1
          for (int u = q0; u < q1; u += 32) {
            pair_weights(u + lane, w0, w1);
            s += w0 + w1;
          }
          s = smp_warp_sum(s);
          if (lane == 0) sm.wtot[0][warp] = s;
          __syncthreads();
          uint64_t before = 0;
          for (int i = 0; i < warp; ++i) before += sm.wtot[0][i];
          if (before <= c.target && c.target < before + s) {   // one warp
#pragma unroll 1
            for (int u = q0; u < q1; u += 32) {
              pair_weights(u + lane, w0, w1);
              const uint64_t incl = before + smp_warp_scan(w0 + w1, lane);
              const uint64_t start = incl - w0 - w1;
              const unsigned who =
                  __ballot_sync(0xFFFFFFFFu, start <= c.target && c.target < incl);
              if (who) {
                const bool second = c.target >= start + w0;
                const int src = __ffs(who) - 1;
                const int token = __shfl_sync(
                    0xFFFFFFFFu, first + 2 * (u + lane) + (second ? 1 : 0), src);
                const float logprob = __shfl_sync(
                    0xFFFFFFFFu, smp_log_share(second ? w1 : w0, c.total), src);
                smp_finish(p, row, token, logprob, lane);
                break;
              }
              before = __shfl_sync(0xFFFFFFFFu, incl, 31);
            }
          }
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
  // Sum of what the cluster's warps reported: every warp for itself.
  auto reported = [&](const auto* x) {
    uint64_t v = 0;
    for (int i = lane; i < cs * kSmpWarps; i += 32) v += x[i];
    return smp_warp_sum(v);
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
    __syncthreads();   // (this CTA's own list lay there)
    sm.buf[tid] = key;
    sm.run[tid] = 0;
    __syncthreads();
    int above = 0;
    uint64_t w = 0;
    if (tid < n) {
#pragma unroll 4
      for (int i = 0; i < n; i += 2) {   // (zeros behind the last)
        const ulonglong2 two = *reinterpret_cast<const ulonglong2*>(&sm.buf[i]);
        above += (two.x > key) + (two.y > key);
      }
      w = weight(smp_value(static_cast<uint32_t>(key >> 32)));
      sm.sorted[above] = key;
      sm.run[above] = w;
    }
    __syncthreads();
    if (tid < n) sm.buf[above] = w;   // the weights, in order
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
    uint64_t c1 = 0, m1 = 0;
    for (int r = 0; r < cs; ++r) {
      c1 += *smp_remote(&sm.cnt[tid], r);
      m1 += (static_cast<uint64_t>(*smp_remote(&sm.mhi[tid], r)) << 32) +
            *smp_remote(&sm.mlo[tid], r);
    }
    uint64_t a = c1, b = m1;
    if (tid == 0) sm.hit = -1;
    block_scan(a, b);
    const uint64_t now = by_mass ? b : a, was = now - (by_mass ? m1 : c1);
    if (was < target && target <= now) {   // one thread's, if any
      sm.hit = tid;
      sm.hit_cnt = static_cast<uint32_t>(c1);
      sm.acc_cnt += a - c1;
      sm.acc_mass += b - m1;
    }
    if (tid == kSmpThreads - 1) sm.binned = b;
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
    c.bin0 = m;
    c.bins = bin_scale;
    state = kAfterHist;
  };
  // The same where the list did not do, over a window around an estimate of
  // the cut: from above by the list's count (weight) and the sampled counts
  // below it, or from below by the sampled counts of the tokens that are cut off
  // (their weight together is known), whichever is the surer; four standard
  // deviations either way, and what the bins' widths may hide, but an eighth of
  // what lies below the list at most. Too many tokens in it: over all.
  auto search_gathered = [&](SmpCmd& c, bool by_mass, uint64_t target) {
    search(c, by_mass, target);
    c.gathered = 0;
    const uint64_t in_list = reported(sm.xlmass);
    // pairs of a warp's run for one that was sampled
    const int turns = per / (32 * kSmpSample), odd = per - turns * 32 * kSmpSample;
    const float each_one = static_cast<float>(per) / (turns * 32 + min(odd, 32));
    uint32_t seen = 0;
    for (int r = 0; r < cs; ++r) seen += *smp_remote(&sm.sampled[tid], r);
    const float count = static_cast<float>(seen) * each_one;
    // a bin's tokens, and their weight in units of 2^24; a list that is
    // complete stands for the bins that it covers
    const int n = sm.list_all, list_bin = n <= kSmpList ? logit_bin(tau_l) : -1;
    const float each_weight = static_cast<float>(weight(m) >> 24) *
                              tc::ex2(-43.0f / (kSmpBins - 0.5f) * (tid + 0.5f));
    const float mid = each_weight * count;
    const uint64_t a0 = tid < list_bin ? 0 : tid == list_bin ? n : static_cast<uint64_t>(count);
    const uint64_t b0 =
        tid < list_bin ? 0 : tid == list_bin ? in_list >> 24 : static_cast<uint64_t>(mid);
    // variance of the sampled weights (counts have their number's)
    const float spread = tid > list_bin ? each_weight * each_weight * count * each_one : 0.0f;
    constexpr int kCountBits = 22;
    const uint64_t own = b0 << kCountBits | a0, own_var = static_cast<uint64_t>(spread);
    uint64_t both = own, var = own_var;
    if (tid == 0) {
      sm.hit = sm.hit2 = kSmpBins - 1;
      sm.over = 0;
      sm.sigma2[0] = sm.sigma2[1] = INFINITY;
    }
    block_scan(both, var);
    const uint64_t whole = smp_warp_sum(lane < kSmpWarps ? sm.wtot[0][lane] : 0) >> kCountBits;
    const uint64_t all_var = smp_warp_sum(lane < kSmpWarps ? sm.wtot[1][lane] : 0);
    const uint64_t a = both & ((1u << kCountBits) - 1u), b = both >> kCountBits;
    const uint64_t now = by_mass ? b : a, was = now - (by_mass ? b0 : a0);
    const uint64_t base = list_bin < 0 ? 0 : by_mass ? in_list >> 24 : n;
    const uint64_t goal_above = by_mass ? target >> 24 : target;
    const uint64_t off = (sm.mass_all - (by_mass ? target : 0)) >> 24;   // cut off
    const uint64_t goal_below = by_mass && whole > off ? whole - off : 0;
    if (was < goal_above && goal_above <= now)
      sm.sigma2[0] = by_mass ? static_cast<float>(var) : each_one * static_cast<float>(now);
    if (was < goal_below && goal_below <= now)
      sm.sigma2[1] = static_cast<float>(all_var - var + own_var);
    __syncthreads();
    const bool below = sm.sigma2[1] < sm.sigma2[0];
    const uint64_t goal = below ? goal_below : goal_above;
    const float rest = goal > base ? static_cast<float>(goal - base) : 0.0f;
    const float part = below ? static_cast<float>(off) : rest;
    const uint64_t slack =
        static_cast<uint64_t>(fminf(rest / 8, 4 * sqrtf(sm.sigma2[below]) + part / 48)) + 2;
    const uint64_t first_goal = goal > base + slack ? goal - slack : base + 1;
    if (was < first_goal && first_goal <= now) {
      sm.hit2 = tid;
      sm.need = a - a0;
    }
    if ((was < goal + slack && goal + slack <= now) ||
        (tid == kSmpThreads - 1 && now < goal + slack)) {
      sm.hit = tid;
      sm.hit_cnt = static_cast<uint32_t>(a);
    }
    if (tid == kSmpThreads - 1 && now < first_goal) sm.need = a - a0;
    __syncthreads();
    const int64_t room = kSmpGathered * kSmpWarps * cs * 4 / 5;
    const int64_t inside = static_cast<int64_t>(sm.hit_cnt) - static_cast<int64_t>(sm.need);
    // (the list's weight is known: a window up to it costs no weights above it)
    c.under_list = list_bin >= 0 && static_cast<int64_t>(sm.hit_cnt) - n < room;
    if (c.under_list || inside < room) {
      c.op = kOpCompact;
      c.gathered = 1;
      // (finite, so that -inf stays below: 513 bins are 29.9 T, beyond float32
      // for temperatures above 1.1e37)
      c.from = fmaxf(m - static_cast<float>(sm.hit + 2) / bin_scale, -3.4028235e38f);
      c.upto = sm.hit2 > 1
                   ? fmaxf(m - static_cast<float>(sm.hit2 - 1) / bin_scale, -3.4028235e38f)
                   : INFINITY;
      if (list_bin >= 0) c.upto = c.under_list ? tau_l : fminf(c.upto, tau_l);
      c.from = fminf(c.from, c.upto);
      c.bin0 = fminf(c.upto, m);
      c.bins = (kSmpBins - 0.5f) / (c.bin0 - c.from);
    }
    __syncthreads();
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
      const uint64_t w = sm.buf[tid];
      uint64_t before = 0;
#pragma unroll 4
      for (int i = 0; i < keep; ++i)
        before += ~static_cast<uint32_t>(sm.sorted[i]) < mine ? sm.buf[i] : 0;
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
        if (!by_k && !by_p) {   // no cut: every key is above it
          if (tid == 0) sm.cut_key = sm.cut_index = 0;
          pick(c);
          return;
        }
        const uint64_t a = reported(sm.xsum);
        if (tid == 0) {
          sm.mass = sm.mass_all = a;
          sm.cut_key = sm.cut_index = 0;
          int n = 0;
          for (int r = 0; r < cs; ++r) n += sm.xlist[r];
          sm.list_all = n;
        }
        __syncthreads();
        const uint64_t goal = by_k ? static_cast<uint64_t>(sm.top_k) : share(sm.mass);
        const uint64_t l = by_groups ? 0 : reported(sm.xlmass);
        // (a list of too few tokens, or too little weight, need not be sorted)
        if ((by_groups || (by_k ? sm.list_all >= sm.top_k : l >= goal)) && from_list())
          c.op = kOpDone;
        else if (by_groups)   // more equal tokens than the list holds
          search(c, false, goal);
        else
          search_gathered(c, !by_k, goal);
        return;
      }
      case kAfterHist:
        if (c.gathered) {
          // what lies above the window comes first
          const uint64_t a = reported(sm.xcnt), b = reported(sm.xsum);
          if (tid == 0) {
            sm.acc_cnt = c.under_list ? sm.list_all : a;
            sm.acc_mass = b;
          }
          __syncthreads();
          bool in = sm.over == 0 && sm.target > (sm.by_mass ? sm.acc_mass : sm.acc_cnt);
          if (in) {
            locate();
            in = sm.hit >= 0;
          }
          if (!in) {   // too many, or the cut is not in the window
            c.gathered = 0;
            search(c, sm.by_mass, sm.target);
            return;
          }
        } else {
          locate();
        }
        if (sm.hit < 0) {   // fewer than top_k tokens have a weight
          __syncthreads();
          if (tid == 0) sm.mass = sm.binned;
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
        c.shift = max(0, 32 - __clz(span) - kSmpBinBits);
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
        if (by_groups) search(c, true, share(sm.mass));
        else search_gathered(c, true, share(sm.mass));
        return;
      }
      // (tokens above the window may be cut by min-p: then over all)
      if (!(tau_0 <= c.from)) c.gathered = 0;
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

constexpr int kSmpFixed = static_cast<int>((sizeof(SmpSmem) + 127) / 128 * 128);
// Rows are cut so that two CTAs fit an SM of 228 KB, 1 KB of each CTA's reserved
// (one's passes run while the other's row arrives: 1024 rows of 154600, normal
// logits of deviation 2, top-p 0.95: 1501 us by eight such, by four that fill an
// SM each 1728; without a cut 454 and 450).
constexpr int kSmpSliceBytes = (228 * 1024 / 2 - 1024 - kSmpFixed) / 16 * 16;
// The longest slice, with a head's and a tail's vector: of float32 by sixteen CTAs.
constexpr int kSmpMostBytes =
    ((kSmpMaxVocab / 4 + 2 + kSmpMaxCluster - 1) / kSmpMaxCluster + 2) * 16;
static_assert(kSmpSliceBytes <= kSmpMostBytes && kSmpFixed + kSmpMostBytes <= 227 * 1024,
              "a slice fits an SM");
static_assert(kSmpSliceBytes / 2 <= 1 << 16 && kSmpMostBytes / 4 <= 1 << 16,
              "gathered places are 16-bit (longer slices than kSmpSliceBytes are float32)");

template <typename T>
dfv_status sample_launch(SampleParams p, cudaStream_t stream) {
  constexpr int kV = SmpVec<T>::kN;
  const int64_t vecs = p.vocab / kV + 2;
  // Few rows over as many CTAs as leave each 4096 tokens at least. Sixteen, which
  // lie in one GPC, for a handful of rows alone (4 rows of 151936 as above: 39 us,
  // by eight 45; 8 rows 48 and 45), eight and four as long as two CTAs an SM hold
  // them all (23 rows: 57, by four 63; 65 rows of 32000 by four 41, by one 58).
  // Not all of such clusters fit at the limits themselves: 37 rows take 91, by
  // four 80, 75 rows of 32000 65, by one 58.
  const int most = p.n_rows <= 4 ? 16 : p.n_rows <= 37 ? 8 : p.n_rows <= 75 ? 4 : 1;
  int cs = 1;
  auto slice = [&]() { return (vecs + cs - 1) / cs + 2; };   // head and tail vectors beside
  while (cs < kSmpMaxCluster &&
         (slice() * 16 > kSmpSliceBytes || (cs < most && p.vocab > cs * 8192)))
    cs <<= 1;
  const int smem = kSmpFixed + static_cast<int>(slice()) * 16;
  static std::atomic<int> allowed[64];   // per device
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return DFV_ERR_CUDA;
  if (!allowed[dev].load(std::memory_order_acquire)) {
    if (cudaFuncSetAttribute(sample_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kSmpFixed + kSmpMostBytes) != cudaSuccess ||
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
