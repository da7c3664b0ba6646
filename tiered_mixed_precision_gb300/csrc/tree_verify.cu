// Which of a tree's drafted tokens are kept, and the token after them.
// (The pages decode one token at a time; FADE-zh §核心机制 fixes the cache that the kept ones join.)
//
// Mathematics: a token is drawn from the target's distribution p after the last kept node, by way of its
// children, which the drafter drew from q. The first child x is kept with probability min(1, p(x) / q(x));
// one that is refused leaves the residual distribution max(p - q, 0), normalised, to the next child, and
// so on; when no child is kept the token is drawn from what is left. Unnormalised, the residual after k
// refusals is r_k = max(p - a_k q, 0) with mass W_k: a_0 = 0, W_0 = 1, a_k+1 = a_k + W_k, so every
// refusal is one more sum over the vocabulary and a child is kept if u q(x) W_k < r_k(x). Drafts without
// probabilities of their own (q is 1 at x) leave p without the refused tokens: kept if u W_k < p(x),
// W_k+1 = W_k - p(x). The final draw is the largest r(i) / E_i with E_i given exponential variates (the
// first of independent arrivals at rates r), greedy rows take the largest logit.
//
// p(i) = 2^((x_i - M) c - log2 S) in fp32 with c = log2(e) / temperature and M the row's maximum. The
// difference comes first: x_i c - M c would lose the last bits of M c, and u q W < r compares p itself,
// so that low temperatures, or logits far from 0, would decide by what was lost. Sums are fp32, in one fixed
// order. A row with NaN or +inf (its sum says so) is gone over again with those replaced.
//
// What bounds it: only nodes on the kept path are looked at, one after another, so a row is a chain of
// passes over its vocabulary. A cluster of CTAs takes a row, each a share of the vocabulary; sums and
// maxima are exchanged through distributed shared memory, and every CTA then decides the same from the
// same numbers. Where all nodes' logits are little to read, their maxima and sums are taken in one pass
// at the start, which leaves the chain one exchange. A pass costs its vectors (words come by asynchronous
// copies, several vectors ahead: 100 us from registers, 77 so, at 64 trees of 128256 tokens) and 2 to 4 us
// of reduction, exchange and waiting for the cluster's slowest: 64 trees of 16 nodes 66 us, 16 chains of 8
// nodes over 50257 tokens 21 us, one greedy chain of 5 over 32000 10 us, of which a launch is half.
#include <cuda_bf16.h>
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "tree.cuh"

namespace fade {
namespace {

// A row's CTAs, their threads and warps. At 64 rows of 128256 tokens 77 us (66 since, by other steps),
// and with 4 CTAs of 512 the same; 8 of 512 (which leave a row waiting for its place) 94, 2 of 512 or
// 1024 and 4 of 1024 from 96 to 99.
constexpr int kCluster = 8, kThreads = 256, kWarps = kThreads / 32;
constexpr int kBatch = 16;    // values exchanged at once
static_assert(kBatch <= 2 * kCluster && (kWarps & (kWarps - 1)) == 0 && kWarps <= 32, "hand_out, over");
constexpr int kNodes = FADE_TREE_MAX_NODES + 1;   // the root first
// All nodes are looked at ahead where a row has at most kAheadLogits of them (nodes x vocabulary, the
// drafter's too), all rows kAheadBytes. us ahead / not, replayed, by a row's logits in M (of trees, fewer
// nodes are kept):
//   1 row    chains: greedy 0.16 10.4 / 16.4, 0.64 16.5 / 22.7; sampled 0.51 16.5 / 14.5, 0.77 24.6 / 24.7,
//            2.05 36.9 / 22.6; certain 0.40 16.5 / 16.5, 1.03 24.7 / 20.6
//            trees: greedy 2.05 24.7 / 12.3; sampled 1.02 22.6 / 14.5; certain 0.51 16.5 / 12.5, 2.05 35 / 21
//   16 rows  chains: sampled 0.51 18.5 / 28.8; certain 0.40 19.5 / 31, 1.03 30.8 / 39.0
//            trees: greedy 0.51 16.6 / 16.5; sampled 1.02 28.8 / 22.6; certain 0.51 20.6 / 20.6
//   64 rows  sampled chains 0.51 33 / 41, trees 0.26 31 / 33, 1.02 51 / 34; 128 rows, chains 0.26 44 / 43.5
// So the rule has a price where logits alone do not tell: 2 to 4 us for one row's sampled chain or certain
// tree of 0.51, 8 us for 16 rows' certain chains of 1.03. Rows and mode would have to be in it.
constexpr long long kAheadLogits = 3 << 18, kAheadBytes = 128ll << 20;
constexpr float kLog2e = 1.4426950408889634f;

struct Args {
  const int32_t *parents, *n_nodes, *tokens;
  const char *target, *target_root, *draft, *draft_root;   // target_root NULL: node 0 is certain
  int64_t t_row, t_node, tr_row, d_row, d_node, dr_row;    // bytes
  const float *temperature, *u, *noise;
  int32_t *path, *n_path, *next;
  int T, V, greedy;   // greedy: every row
  int ahead;          // all nodes are looked at in one pass, kBatch of them a time
};

// A logit as it counts: NaN reads as -inf, +inf as the largest number.
__device__ __forceinline__ float logit(float x) {
  return x != x ? -INFINITY : fminf(x, 3.402823466e38f);
}
__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }

// 16 bytes of consecutive elements; `wide`: they start on a 16-byte boundary.
template <typename E>
struct Vec {
  static constexpr int N = 16 / sizeof(E);
};
template <typename E>
union Words {
  uint4 w;
  E e[Vec<E>::N];
  __device__ __forceinline__ Words() {}
};
template <typename E>
__device__ __forceinline__ void load(const E* x, int i, bool wide, Words<E>& v) {
  if (wide) {
    v.w = __ldg(reinterpret_cast<const uint4*>(x + i));
  } else {
#pragma unroll
    for (int j = 0; j < Vec<E>::N; ++j) v.e[j] = x[i + j];
  }
}
template <typename E>
__device__ __forceinline__ void logits(const Words<E>& v, bool careful, float (&y)[Vec<E>::N]) {
#pragma unroll
  for (int j = 0; j < Vec<E>::N; ++j) y[j] = to_float(v.e[j]);
  if (careful) {
#pragma unroll
    for (int j = 0; j < Vec<E>::N; ++j) y[j] = logit(y[j]);
  }
}

// The largest of a vector's elements (x: the same, as `logits` gives them); NaN only if all are.
template <typename E>
__device__ __forceinline__ float top_of(const Words<E>& w, bool careful, const float (&x)[Vec<E>::N]) {
  if (sizeof(E) == 4 || careful) {
    float top = x[0];
#pragma unroll
    for (int j = 1; j < Vec<E>::N; ++j) top = fmaxf(top, x[j]);
    return top;
  }
  if constexpr (sizeof(E) == 2) {   // two elements an instruction
    using E2 = typename std::conditional<std::is_same<E, __half>::value, __half2, __nv_bfloat162>::type;
    const E2* e = reinterpret_cast<const E2*>(&w.w);
    const E2 m = __hmax2(__hmax2(e[0], e[1]), __hmax2(e[2], e[3]));
    return fmaxf(to_float(m.x), to_float(m.y));
  }
  return 0.f;
}

// ---------------------------------------------------------------- cluster
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile(
      "barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t remote(const void* p, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
}
__device__ __forceinline__ void st_remote4(uint32_t at, float4 v) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(at), "f"(v.x), "f"(v.y),
               "f"(v.z), "f"(v.w)
               : "memory");
}
__device__ __forceinline__ void st_remote(uint32_t at, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(at), "r"(v) : "memory");
}

// Kinds of values that are reduced, up to four floats each: two joined, a warp's (over groups of `width`
// lanes, in all of which it ends), or the CTAs' of a cluster in their order. Maxima come first and every
// sum is scaled once (scaled at each of a warp's five steps: 74 us at 64 trees, 66 now).
__device__ __forceinline__ float other(float x, int o) { return __shfl_xor_sync(~0u, x, o); }
template <bool TWO>
struct Stats {   // maximum and sum of 2^((x - maximum) c), of the target and (TWO) the drafter
  float c;
  __device__ __forceinline__ float share(float m, float top) const {   // of a sum that goes with m
    return top == -INFINITY ? 1.f : ex2((m - top) * c);                // (all empty, sums of 0)
  }
  __device__ __forceinline__ void join(float& m, float& s, float m2, float s2) const {
    const float n = fmaxf(m, m2);
    s = s * share(m, n) + s2 * share(m2, n);
    m = n;
  }
  __device__ __forceinline__ float4 operator()(float4 a, float4 b) const {
    join(a.x, a.y, b.x, b.y);
    if (TWO) join(a.z, a.w, b.z, b.w);
    return a;
  }
  __device__ __forceinline__ float4 over(float4 v, int width) const {
    float m = v.x, n = v.z;
    for (int o = width / 2; o; o >>= 1) {
      m = fmaxf(m, other(m, o));
      if (TWO) n = fmaxf(n, other(n, o));
    }
    v.y *= share(v.x, m);
    if (TWO) v.w *= share(v.z, n);
    for (int o = width / 2; o; o >>= 1) {
      v.y += other(v.y, o);
      if (TWO) v.w += other(v.w, o);
    }
    v.x = m;
    v.z = n;
    return v;
  }
  __device__ __forceinline__ float4 all(const float4 (&v)[kCluster]) const {
    float4 r = v[0];
#pragma unroll
    for (int i = 1; i < kCluster; ++i) {
      r.x = fmaxf(r.x, v[i].x);
      if (TWO) r.z = fmaxf(r.z, v[i].z);
    }
    r.y *= share(v[0].x, r.x);
    if (TWO) r.w *= share(v[0].z, r.z);
#pragma unroll
    for (int i = 1; i < kCluster; ++i) {
      r.y += v[i].y * share(v[i].x, r.x);
      if (TWO) r.w += v[i].w * share(v[i].z, r.z);
    }
    return r;
  }
};
struct Sum {
  __device__ __forceinline__ float4 over(float4 v, int width) const {
    for (int o = width / 2; o; o >>= 1) v.x += other(v.x, o);
    return v;
  }
  __device__ __forceinline__ float4 all(const float4 (&v)[kCluster]) const {
    float4 r = v[0];
#pragma unroll
    for (int i = 1; i < kCluster; ++i) r.x += v[i].x;
    return r;
  }
};
struct Best {   // the larger value, the lower index where they are equal (y: the index's bits)
  __device__ __forceinline__ float4 operator()(float4 a, float4 b) const {
    const bool take = b.x > a.x || (b.x == a.x && __float_as_int(b.y) < __float_as_int(a.y));
    return take ? b : a;
  }
  __device__ __forceinline__ float4 over(float4 v, int width) const {
    for (int o = width / 2; o; o >>= 1)
      v = (*this)(v, make_float4(other(v.x, o), other(v.y, o), 0.f, 0.f));
    return v;
  }
  __device__ __forceinline__ float4 all(const float4 (&v)[kCluster]) const {
    float4 r = v[0];
#pragma unroll
    for (int i = 1; i < kCluster; ++i) r = (*this)(r, v[i]);
    return r;
  }
};

struct Shared {
  float4 warps[kBatch][kWarps];
  float4 ranks[2][kBatch][kCluster];   // what each CTA of the cluster found, two calls in turn
  float4 stats[kNodes];                // of node i - 1
  uint64_t kids[kNodes];               // children of node i - 1
  // from CTA 0, the same in all: per node its parent, token, uniform number, its target and drafter
  // logits after its parent; then nodes, temperature
  int32_t parent[FADE_TREE_MAX_NODES], token[FADE_TREE_MAX_NODES];
  float u[FADE_TREE_MAX_NODES], tl[FADE_TREE_MAX_NODES], ql[FADE_TREE_MAX_NODES];
  int32_t n;
  float temperature;
  int32_t refused[FADE_TREE_MAX_NODES];
};

// A thread's value joined over its warp, kept as the i-th.
template <class Op>
__device__ __forceinline__ void keep(Shared& sh, int i, float4 v, const Op& op) {
  v = op.over(v, 32);
  if ((threadIdx.x & 31) == 0) sh.warps[i][threadIdx.x >> 5] = v;
}
// The values 0 .. count - 1 joined over the whole cluster, from then on in sh.ranks (exchanged).
template <class Op>
__device__ __forceinline__ void exchange(Shared& sh, int count, const Op& op, int& turn) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t rank = cluster_rank();
  __syncthreads();
  for (int i = warp; i < count; i += kWarps) {   // (every eight lanes have all of them)
    const float4 v = op.over(sh.warps[i][lane & (kWarps - 1)], kWarps);
    if (lane < kCluster) st_remote4(remote(&sh.ranks[turn][i][rank], lane), v);
  }
  cluster_sync();
  turn ^= 1;
}
template <class Op>
__device__ __forceinline__ float4 exchanged(const Shared& sh, int i, const Op& op, int turn) {
  return op.all(sh.ranks[turn ^ 1][i]);
}
// The i-th value of this CTA, whole as it is, handed to every CTA as the cluster's to[i], i < count <= 2.
template <class Op>
__device__ __forceinline__ void hand_out(Shared& sh, int count, int first, int apart, const Op& op,
                                         int& turn) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  __syncthreads();
  if (warp < count) {
    const float4 v = op.over(sh.warps[warp][lane & (kWarps - 1)], kWarps);
    if (lane < kCluster) st_remote4(remote(&sh.ranks[turn][first + warp * apart][0], lane), v);
  }
  cluster_sync();
  turn ^= 1;
}
template <class Op>
__device__ __forceinline__ float4 reduce(Shared& sh, float4 v, const Op& op, int& turn) {
  keep(sh, 0, v, op);
  exchange(sh, 1, op, turn);
  return exchanged(sh, 0, op, turn);
}

// ---------------------------------------------------------------- passes over the vocabulary
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ uint4 ld_shared16(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(at)
               : "memory");
  return v;
}

// The logits after a node.
template <typename E>
struct Node {
  const E *t, *d;
  int head;         // elements before the first 16-byte boundary of t
  bool wide_d;      // d has the same boundaries
};

constexpr int kSlots = 8;   // 16-byte words of a thread that copies are in flight to

// A row and a thread's share of it.
template <typename E, bool DRAFT>
struct Row {
  static constexpr int N = Vec<E>::N;
  const Args& a;
  int b, first, step;             // the row; the thread's vectors
  uint32_t slot0;                 // its slots: kThreads words apart
  static constexpr uint32_t slot_bytes = kThreads * 16;
  __device__ __forceinline__ Node<E> node_at(int node) const {   // (-1: the root)
    Node<E> x;
    x.t = reinterpret_cast<const E*>(node < 0 ? a.target_root + b * a.tr_row
                                              : a.target + b * a.t_row + node * a.t_node);
    x.d = !DRAFT ? nullptr
                 : reinterpret_cast<const E*>(node < 0 ? a.draft_root + b * a.dr_row
                                                       : a.draft + b * a.d_row + node * a.d_node);
    x.head = min((int)((16 - (reinterpret_cast<uintptr_t>(x.t) & 15)) & 15) / (int)sizeof(E), a.V);
    x.wide_d = DRAFT && (reinterpret_cast<uintptr_t>(x.d + x.head) & 15) == 0;
    return x;
  }
  // One pass over the logits after node `at`, then those after then(at), .., `most` nodes (-2: no more).
  // f(index, W words of t, of d, noise) for a thread's vectors, g(index, t, d, noise) for single elements
  // at the ends, done(k) after the k-th node. D, NOISE: d and the noise are read, too (W = 1). Words come
  // by asynchronous copies into slots of the thread's own, several vectors ahead, across nodes.
  template <bool D, bool NOISE, int W, class Then, class F, class G, class Done>
  __device__ __forceinline__ void sweep(int at, int most, const Then& then, const F& f, const G& g,
                                        const Done& done) const {
    constexpr int EW = NOISE ? N / 4 : 0;               // words of noise a vector
    constexpr int P = W * (1 + (D ? 1 : 0)) + EW;       // words of a vector
    constexpr int S = P == 1 ? 8 : P == 2 ? 4 : 2;      // vectors in flight
    static_assert(P * S <= kSlots && (W == 1 || !NOISE), "slots");
    auto vecs_of = [&](const Node<E>& x) { return (a.V - x.head) / (W * N); };
    const float* noise = NOISE && a.noise ? a.noise + (size_t)b * a.V : nullptr;
    auto wide_e = [&](const Node<E>& x) {
      return noise && (reinterpret_cast<uintptr_t>(noise + x.head) & 15) == 0;
    };
    int ai = at, ki = 0, vi = first;
    Node<E> ni = node_at(at);
    int vecs_i = vecs_of(ni);
    uint32_t si = 0, sp = 0;
    auto issue = [&]() {
      while (ai != -2 && vi >= vecs_i) {
        ai = ++ki < most ? then(ai) : -2;
        if (ai == -2) break;
        ni = node_at(ai);
        vecs_i = vecs_of(ni);
        vi = first;
      }
      if (ai != -2) {
        const int i = ni.head + vi * (W * N);
        const uint32_t to = slot0 + si * P * slot_bytes;
#pragma unroll
        for (int w = 0; w < W; ++w) copy16(to + w * slot_bytes, ni.t + i + w * N);
        if (D && ni.wide_d) {
#pragma unroll
          for (int w = 0; w < W; ++w) copy16(to + (W + w) * slot_bytes, ni.d + i + w * N);
        }
        if (NOISE && wide_e(ni)) {
#pragma unroll
          for (int k = 0; k < EW; ++k) copy16(to + (P - EW + k) * slot_bytes, noise + i + 4 * k);
        }
        vi += step;
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
      si = si + 1 == S ? 0 : si + 1;
    };
#pragma unroll 1
    for (int i = 0; i < S; ++i) issue();
#pragma unroll 1
    for (int k = 0; at != -2; at = ++k < most ? then(at) : -2) {
      const Node<E> node = node_at(at);
      const int vecs = vecs_of(node);
#pragma unroll 1
      for (int v = first; v < vecs; v += step) {
        const int i = node.head + v * (W * N);
        const uint32_t from = slot0 + sp * P * slot_bytes;
        Words<E> t[W], d[W];
        float e[N];
        asm volatile("cp.async.wait_group %0;" ::"n"(S - 1) : "memory");
#pragma unroll
        for (int w = 0; w < W; ++w) t[w].w = ld_shared16(from + w * slot_bytes);
        if (D) {
#pragma unroll
          for (int w = 0; w < W; ++w)
            if (node.wide_d)
              d[w].w = ld_shared16(from + (W + w) * slot_bytes);
            else
              load(node.d, i + w * N, false, d[w]);
        }
        if (NOISE) {
          if (wide_e(node)) {
#pragma unroll
            for (int q = 0; q < EW; ++q) {
              const uint4 z = ld_shared16(from + (P - EW + q) * slot_bytes);
              e[4 * q] = __uint_as_float(z.x), e[4 * q + 1] = __uint_as_float(z.y);
              e[4 * q + 2] = __uint_as_float(z.z), e[4 * q + 3] = __uint_as_float(z.w);
            }
          } else {
#pragma unroll
            for (int q = 0; q < N; ++q) e[q] = noise ? noise[i + q] : 1.f;
          }
        }
        issue();
        sp = sp + 1 == S ? 0 : sp + 1;
        f(i, t, d, e);
      }
      const int ends = a.V - vecs * (W * N);
      if (first < ends) {
        const int i = first < node.head ? first : first + vecs * (W * N);
        g(i, logit(to_float(node.t[i])), D ? logit(to_float(node.d[i])) : 0.f,
          NOISE && noise ? noise[i] : 1.f);
      }
      done(k);
    }
  }
};

// The distributions after a node. p(i) = 2^((x_i - mt) c + lt), a q(i) = 2^((y_i - md) c + ld + la); an empty
// row's are 2^-inf. Where p and q are the same numbers, p - 1 q is nothing to the last bit. careful: the
// logits have NaN or infinities.
template <typename E, bool DRAFT>
struct Probs {
  static constexpr int N = Vec<E>::N;
  float c, mt, md, lt, ld;
  float taken, la;   // a, log2 a
  bool careful;
  __device__ __forceinline__ float p_of(float x) const { return ex2(fmaf(x - mt, c, lt)); }
  __device__ __forceinline__ float q_of(float y, float l) const { return ex2(fmaf(y - md, c, ld + l)); }
  __device__ __forceinline__ float r_of(float x, float y) const {
    const float p = p_of(x);
    return DRAFT && taken > 0.f ? fmaxf(p - q_of(y, la), 0.f) : p;
  }
  // r of a vector, two elements an instruction (the same bits as r_of's)
  template <bool Q>
  __device__ __forceinline__ void rest(const Words<E>& t, const Words<E>& d, float (&r)[N]) const {
    float x[N], y[N];
    logits(t, careful, x);
    if constexpr (Q) logits(d, careful, y);
    const f2x c2 = f2_pack(c, c), mt2 = f2_pack(mt, mt), lt2 = f2_pack(lt, lt);
    const f2x md2 = f2_pack(md, md), ld2 = f2_pack(ld + la, ld + la);
#pragma unroll
    for (int j = 0; j < N; j += 2) {
      f2_unpack(f2_fma(f2_sub(f2_pack(x[j], x[j + 1]), mt2), c2, lt2), r[j], r[j + 1]);
      r[j] = ex2(r[j]);
      r[j + 1] = ex2(r[j + 1]);
      if constexpr (Q) {
        float q[2];
        f2_unpack(f2_fma(f2_sub(f2_pack(y[j], y[j + 1]), md2), c2, ld2), q[0], q[1]);
        r[j] = fmaxf(r[j] - ex2(q[0]), 0.f);
        r[j + 1] = fmaxf(r[j + 1] - ex2(q[1]), 0.f);
      }
    }
  }
};

template <typename E, bool DRAFT, bool AHEAD>
__global__ void __launch_bounds__(kThreads, 4) tree_verify_kernel(const __grid_constant__ Args a) {
  constexpr int N = Vec<E>::N;
  __shared__ Shared sh;
  extern __shared__ uint4 slots[];   // [kSlots][threads]
  const int tid = threadIdx.x;
  const uint32_t rank = cluster_rank();
  constexpr int size = kCluster;
  const int b = blockIdx.x / size;
  const Row<E, DRAFT> row{a, b, (int)(rank * kThreads + tid), (int)(size * kThreads),
                          smem_u32(slots + tid)};
  int turn = 0;
  // (waited for before the first write to another CTA, which has to have started by then)
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");

  auto stop = [](int) { return -2; };
  auto nothing = [](int) {};

  // a thread's share of rows' maxima and sums, or of their greatest logits (greedy): kept as the 0th, 1st, ..
  const Best best_of;
  const float4 none = make_float4(0.f, __int_as_float(0x7fffffff), 0.f, 0.f);
  auto look = [&](const Row<E, DRAFT>& row, int at, int most, auto then, bool greedy, float c,
                  bool careful) {
    const Stats<DRAFT> join{c};
    if (greedy) {
      float4 best = none;
      best.x = -INFINITY;
      row.template sweep<false, false, 2>(   // (two words a vector: 12.4 -> 10.4 us at a chain of 5)
            at, most, then,
            [&](int i, const Words<E>(&t)[2], const Words<E>(&)[2], const float(&)[N]) {
              float x[2 * N];
#pragma unroll
              for (int j = 0; j < 2 * N; ++j) x[j] = to_float(t[j / N].e[j % N]);
              float top = x[0];
#pragma unroll
              for (int j = 1; j < 2 * N; ++j) top = fmaxf(top, x[j]);
              if (top > best.x) {   // (ascending in a thread)
#pragma unroll
                for (int j = 0; j < 2 * N; ++j)
                  if (logit(x[j]) > best.x)
                    best = make_float4(logit(x[j]), __int_as_float(i + j), 0.f, 0.f);
              }
            },
            [&](int i, float x, float, float) {
              if (x > -INFINITY) best = best_of(best, make_float4(x, __int_as_float(i), 0.f, 0.f));
            },
            [&](int k) {
              keep(sh, k, best, best_of);
              best = none;
              best.x = -INFINITY;
            });
      return;
    }
    float4 st = make_float4(-INFINITY, 0.f, -INFINITY, 0.f);
    auto add = [&](float& m, float& s, const Words<E>& w) {
      float x[N];
      logits(w, careful, x);
      const float top = top_of(w, careful, x);
      if (top > m) {
        s *= ex2((m - top) * c);   // (0 from -inf)
        m = top;
      }
      if (m == -INFINITY) {   // nothing above -inf so far; NaN has to show in the sum all the same
        float any = x[0];
#pragma unroll
        for (int j = 1; j < N; ++j) any += x[j];
        if (any != any) s = any;
        return;
      }
      const f2x c2 = f2_pack(c, c), m2 = f2_pack(m, m);
      f2x sum = f2_pack(0.f, 0.f);
#pragma unroll
      for (int j = 0; j < N; j += 2) {
        float y0, y1;
        f2_unpack(f2_mul(f2_sub(f2_pack(x[j], x[j + 1]), m2), c2), y0, y1);
        sum = f2_add(sum, f2_pack(ex2(y0), ex2(y1)));
      }
      float s0, s1;
      f2_unpack(sum, s0, s1);
      s += s0 + s1;
    };
    row.template sweep<DRAFT, false, 1>(
          at, most, then,
          [&](int, const Words<E>(&t)[1], const Words<E>(&d)[1], const float(&)[N]) {
            add(st.x, st.y, t[0]);
            if (DRAFT) add(st.z, st.w, d[0]);
          },
          [&](int, float x, float y, float) {
            st = join(st, make_float4(x, x == -INFINITY ? 0.f : 1.f, DRAFT ? y : -INFINITY,
                                      DRAFT && y != -INFINITY ? 1.f : 0.f));
          },
          [&](int k) {
            keep(sh, k, st, join);
            st = make_float4(-INFINITY, 0.f, -INFINITY, 0.f);
          });
  };
  auto scale_of = [](float temp) { return kLog2e / fminf(fmaxf(temp, 1e-30f), 1e30f); };
  auto in_line = [&](int at) { return at + 1 < a.T ? at + 1 : -2; };
  constexpr int most = AHEAD ? kBatch : 1;
  // Several nodes at once: a CTA takes whole ones, whose values are joined once and not in every CTA
  // (16 chains of 8 nodes, 50257 tokens: 28.8 us without, 22 with).
  const Row<E, DRAFT> alone{a, b, tid, kThreads, smem_u32(slots + tid)};

  // The first nodes' pass needs nothing of the tree but the temperature; CTA 0 hands out the rest
  // meanwhile, and what every CTA decides by is what CTA 0 read.
  int cur = a.target_root ? -1 : 0;
  const float own_temp = a.greedy ? 0.f : a.temperature ? a.temperature[b] : 1.f;
  const bool mine = rank == 0 && tid < a.T, last = rank == 0 && tid == kThreads - 1;
  int parent = -1, token = -1, nodes = a.T;
  float tl = -INFINITY, ql = -INFINITY, u = 0.f;
  if (mine) {
    const size_t at = (size_t)b * a.T + tid;
    parent = a.parents[at];
    if (parent < 0 || parent >= tid) parent = -1;
    token = a.tokens[at];
    if (!a.greedy) u = a.u[at];
    if (token >= 0 && token < a.V && (parent >= 0 || a.target_root)) {
      const Node<E> x = row.node_at(parent);
      tl = logit(to_float(x.t[token]));
      if (DRAFT) ql = logit(to_float(x.d[token]));
    }
  } else if (last && a.n_nodes) {
    nodes = min(max(a.n_nodes[b], 0), a.T);
  }
  if (tid < kNodes) sh.kids[tid] = 0;
  uint64_t known = 0;   // nodes whose maxima and sums lie in sh.stats
  bool known_root = false;
  // nodes cur, cur + 1, .. looked at, and their values exchanged
  auto look_on = [&](bool greedy, float c, auto before) {
    const int count = min(most, a.T - cur);
    const Stats<DRAFT> join{c};
    const bool apart = AHEAD && count >= kCluster / 2;
    const int mine = apart ? ((int)rank < count) + ((int)(rank + size) < count) : 0;
    if (!apart)
      look(row, cur, most, in_line, greedy, c, false);
    else if (mine > 0)
      look(alone, cur + rank, mine, [&](int at) { return at + (int)size; }, greedy, c, false);
    before();
    if (greedy) {
      if (apart)
        hand_out(sh, mine, rank, size, best_of, turn);
      else
        exchange(sh, count, best_of, turn);
    } else {
      if (apart)
        hand_out(sh, mine, rank, size, join, turn);
      else
        exchange(sh, count, join, turn);
    }
    if (tid < count)
      sh.stats[cur + 1 + tid] = apart    ? sh.ranks[turn ^ 1][tid][0]
                                : greedy ? exchanged(sh, tid, best_of, turn)
                                         : exchanged(sh, tid, join, turn);
    for (int k = 0; k < count; ++k) {
      if (cur + k < 0)
        known_root = true;
      else
        known |= 1ull << (cur + k);
    }
  };
  look_on(!(own_temp > 0.f), scale_of(own_temp), [&]() {
    __syncwarp();
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    for (int r = 0; r < size; ++r) {
      if (mine) {
        st_remote(remote(&sh.parent[tid], r), parent);
        st_remote(remote(&sh.token[tid], r), token);
        st_remote(remote(&sh.u[tid], r), __float_as_uint(u));
        st_remote(remote(&sh.tl[tid], r), __float_as_uint(tl));
        st_remote(remote(&sh.ql[tid], r), __float_as_uint(ql));
      }
      if (last) {
        st_remote(remote(&sh.n, r), nodes);
        st_remote(remote(&sh.temperature, r), __float_as_uint(own_temp));
      }
    }
  });
  const int n = sh.n;
  const bool greedy = !(sh.temperature > 0.f);
  const float c = scale_of(sh.temperature);
  const Stats<DRAFT> join{c};
  if (tid < n)
    atomicOr(reinterpret_cast<unsigned long long*>(&sh.kids[sh.parent[tid] + 1]), 1ull << tid);
  __syncthreads();
  const bool lead = rank == 0 && tid == 0;

  int kept = 0, next = -1;
  int32_t* path = a.path + (size_t)b * a.T;
  if (!a.target_root && n > 0) {
    if (lead) path[0] = 0;
    kept = 1;
  }
  const bool any = a.target_root || n > 0;   // (no node and no root: nothing to draw from)
  while (any) {
    const uint64_t kids = sh.kids[cur + 1];
    int take = -1;
    if (!(cur < 0 ? known_root : (known >> cur) & 1)) {
      look_on(greedy, c, [] {});
      __syncthreads();
    }
    float4 st = sh.stats[cur + 1];

    if (greedy) {
      const int top = st.x == -INFINITY ? -1 : __float_as_int(st.y);
      for (uint64_t left = kids; left && take < 0; left &= left - 1) {
        const int i = __ffsll((long long)left) - 1;
        if (top >= 0 && sh.token[i] == top) take = i;
      }
      next = top;
    } else {
      const bool careful = !(st.y < INFINITY && st.w < INFINITY);   // (NaN and +inf show in the sums)
      if (careful) {
        look(row, cur, 1, stop, false, c, true);
        exchange(sh, 1, join, turn);
        st = exchanged(sh, 0, join, turn);
      }
      Probs<E, DRAFT> pr;
      pr.c = c;
      pr.mt = st.x == -INFINITY ? 0.f : st.x;
      pr.md = st.z == -INFINITY ? 0.f : st.z;
      pr.lt = st.y > 0.f ? -log2f(st.y) : 0.f;
      pr.ld = st.w > 0.f ? -log2f(st.w) : 0.f;
      pr.taken = pr.la = 0.f;
      pr.careful = careful;
      float left_mass = 1.f;   // W

      // -------------------------------------------- children
      int refused = 0;
      for (uint64_t left = kids; left; left &= left - 1) {
        const int i = __ffsll((long long)left) - 1, x = sh.token[i];
        float r = pr.r_of(sh.tl[i], sh.ql[i]);
        if (!DRAFT)
          for (int j = 0; j < refused; ++j)
            if (sh.refused[j] == x) r = 0.f;
        if (sh.u[i] * (DRAFT ? pr.q_of(sh.ql[i], 0.f) : 1.f) * left_mass < r) {
          take = i;
          break;
        }
        if (DRAFT) {
          pr.taken += left_mass;
          pr.la = log2f(pr.taken);
          if (!(left & (left - 1))) break;   // (the last child: nobody asks for what is left)
          float4 w = make_float4(0.f, 0.f, 0.f, 0.f);
          row.template sweep<DRAFT, false, 1>(
                cur, 1, stop,
                [&](int, const Words<E>(&t)[1], const Words<E>(&d)[1], const float(&)[N]) {
                  float r[N], part[2];
                  pr.template rest<DRAFT>(t[0], d[0], r);
                  f2x sum = f2_pack(r[0], r[1]);
#pragma unroll
                  for (int j = 2; j < N; j += 2) sum = f2_add(sum, f2_pack(r[j], r[j + 1]));
                  f2_unpack(sum, part[0], part[1]);
                  w.x += part[0] + part[1];
                },
                [&](int, float x, float y, float) { w.x += pr.r_of(x, y); }, nothing);
          left_mass = reduce(sh, w, Sum(), turn).x;
        } else {
          left_mass = fmaxf(left_mass - r, 0.f);
          __syncthreads();
          if (tid == 0) sh.refused[refused] = x;
          ++refused;
          __syncthreads();
        }
      }
      if (take < 0) {
        // ------------------------------------------ the draw
        float4 best = none;
        auto race = [&](int i, float r, float e) {
          if (r > best.x * e * 0.999999f && r > 0.f)   // (the quotient only where it may win)
            best = best_of(best, make_float4(r / e, __int_as_float(i), 0.f, 0.f));
        };
        auto draw = [&](auto with_q) {
          constexpr bool Q = decltype(with_q)::value;
          row.template sweep<Q, true, 1>(
                cur, 1, stop,
                [&](int i, const Words<E>(&t)[1], const Words<E>(&d)[1], const float(&e)[N]) {
                  float r[N];
                  pr.template rest<Q>(t[0], d[0], r);
                  if (!DRAFT)
                    for (int k = 0; k < refused; ++k)
                      if ((unsigned)sh.refused[k] - (unsigned)i < (unsigned)N) {
#pragma unroll
                        for (int j = 0; j < N; ++j)
                          if (sh.refused[k] == i + j) r[j] = 0.f;
                      }
#pragma unroll
                  for (int j = 0; j < N; ++j) race(i + j, r[j], e[j]);
                },
                [&](int i, float x, float y, float e) {
                  float r = pr.r_of(x, y);
                  if (!DRAFT)
                    for (int k = 0; k < refused; ++k)
                      if (sh.refused[k] == i) r = 0.f;
                  race(i, r, e);
                },
                nothing);
        };
        while (true) {
          best = none;
          if constexpr (DRAFT) {
            if (pr.taken > 0.f)
              draw(std::true_type());
            else
              draw(std::false_type());
          } else {
            draw(std::false_type());
          }
          best = reduce(sh, best, best_of, turn);
          if (best.x > 0.f || (pr.taken == 0.f && refused == 0)) break;
          pr.taken = 0.f;   // nothing is left (p and q alike to the last bit): p itself
          refused = 0;
        }
        next = best.x > 0.f ? __float_as_int(best.y) : -1;
      }
    }
    if (take < 0) break;
    if (lead) path[kept] = take;
    ++kept;
    cur = take;
  }
  if (rank == 0) {
    if (tid >= kept && tid < a.T) path[tid] = 0;
    if (tid == 0) {
      a.n_path[b] = kept;
      a.next[b] = next;
    }
  }
}

template <typename E, bool DRAFT>
fade_status_t launch(const Args& a, int B, cudaStream_t st) {
  cudaLaunchConfig_t lc{};
  lc.gridDim = dim3(B * kCluster);
  lc.blockDim = dim3(kThreads);
  lc.dynamicSmemBytes = kThreads * kSlots * 16;
  lc.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim = {kCluster, 1, 1};
  lc.attrs = at;
  lc.numAttrs = 1;
  const cudaError_t e = a.ahead ? cudaLaunchKernelEx(&lc, tree_verify_kernel<E, DRAFT, true>, a)
                                : cudaLaunchKernelEx(&lc, tree_verify_kernel<E, DRAFT, false>, a);
  if (e != cudaSuccess)
    return set_error(FADE_ERR_CUDA, "fade_tree_verify: %s", cudaGetErrorString(e));
  return launch_status("fade_tree_verify");
}
template <typename E>
fade_status_t launch(const Args& a, int B, cudaStream_t st) {
  return a.draft ? launch<E, true>(a, B, st) : launch<E, false>(a, B, st);
}

}  // namespace
}  // namespace fade

using namespace fade;

extern "C" fade_status_t fade_tree_verify(const fade_config_t* c, int32_t T, int32_t vocab,
                                          int32_t type, const int32_t* parents,
                                          const int32_t* n_nodes, const int32_t* tokens,
                                          const fade_logits_t* target,
                                          const fade_logits_t* target_root,
                                          const fade_logits_t* draft,
                                          const fade_logits_t* draft_root,
                                          const float* temperature, const float* u,
                                          const float* noise, int32_t* path, int32_t* n_path,
                                          int32_t* next, void* stream) {
  clear_error();
  FADE_RANGE("fade_tree_verify");
  fade_status_t st = validate_tree(c, T);
  if (st) return st;
  if (vocab < 1 || vocab > FADE_MAX_VOCAB)
    return set_error(FADE_ERR_INVALID_ARGUMENT, "vocabulary %d outside [1, %d]", vocab,
                     FADE_MAX_VOCAB);
  if (type < FADE_LOGITS_F16 || type > FADE_LOGITS_F32)
    return set_error(FADE_ERR_INVALID_ARGUMENT, "unknown logit type %d", type);
  if (!parents || !tokens || !path || !n_path || !next)
    return set_error(FADE_ERR_INVALID_ARGUMENT, "NULL parents, tokens, path, n_path or next");
  for (const void* p : {(const void*)parents, (const void*)n_nodes, (const void*)tokens,
                        (const void*)temperature, (const void*)u, (const void*)noise,
                        (const void*)path, (const void*)n_path, (const void*)next})
    if (!aligned(p, 4))
      return set_error(FADE_ERR_INVALID_ARGUMENT, "32-bit arguments must be 4-byte aligned");
  const int size = type == FADE_LOGITS_F32 ? 4 : 2;
  if (!target) return set_error(FADE_ERR_INVALID_ARGUMENT, "NULL target");
  for (const fade_logits_t* x : {target, target_root, draft, draft_root})
    if (x && (!x->x || !aligned(x->x, size)))
      return set_error(FADE_ERR_INVALID_ARGUMENT, "logits are NULL or not aligned to their type");
  if (draft && !u)
    return set_error(FADE_ERR_INVALID_ARGUMENT, "drafter logits need uniform numbers");
  if ((draft && target_root && !draft_root) || (draft_root && !(draft && target_root)))
    return set_error(FADE_ERR_INVALID_ARGUMENT,
                     "drafter logits are needed where target logits are: after the nodes and, where the "
                     "target's are given there, after the last cached token");
  Args a{};
  a.parents = parents;
  a.n_nodes = n_nodes;
  a.tokens = tokens;
  auto at = [](const fade_logits_t* x) { return x ? static_cast<const char*>(x->x) : nullptr; };
  a.target = at(target);
  a.target_root = at(target_root);
  a.draft = at(draft);
  a.draft_root = at(draft_root);
  a.t_row = target->row_stride * size;
  a.t_node = target->node_stride * size;
  a.tr_row = target_root ? target_root->row_stride * size : 0;
  a.d_row = draft ? draft->row_stride * size : 0;
  a.d_node = draft ? draft->node_stride * size : 0;
  a.dr_row = draft_root ? draft_root->row_stride * size : 0;
  a.temperature = temperature;
  a.u = u;
  a.noise = noise;
  a.path = path;
  a.n_path = n_path;
  a.next = next;
  a.T = T;
  a.V = vocab;
  a.greedy = u == nullptr;
  const long long row = (long long)T * vocab * (draft ? 2 : 1);
  a.ahead = row <= kAheadLogits && c->batch * row * size <= kAheadBytes;
  const cudaStream_t s = as_stream(stream);
  if (type == FADE_LOGITS_F16) return launch<__half>(a, c->batch, s);
  if (type == FADE_LOGITS_BF16) return launch<__nv_bfloat16>(a, c->batch, s);
  return launch<float>(a, c->batch, s);
}
