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
// p(i) = 2^((x_i - M) log2(e) / temperature) / S in fp32, M the row's maximum: the largest terms lose
// nothing in the subtraction. Sums are fp32, in one fixed order.
//
// What bounds it: only nodes on the kept path are looked at, one after another, so a row is a chain of
// reads of its vocabulary. A cluster of CTAs takes a row, each a share of the vocabulary; sums and maxima
// are exchanged through distributed shared memory, and every CTA then decides the same from the same
// numbers.
#include <cuda_bf16.h>
#include <math.h>

#include <algorithm>

#include "prompt.cuh"

namespace fade {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kCluster = 8;   // CTAs of a row
constexpr int kUnroll = 4;    // vectors in flight a thread and array
constexpr float kLog2e = 1.4426950408889634f;

struct Args {
  const int32_t *parents, *n_nodes, *tokens;
  const char *target, *target_root, *draft, *draft_root;   // target_root NULL: node 0 is certain
  int64_t t_row, t_node, tr_row, d_row, d_node, dr_row;    // bytes
  const float *temperature, *u, *noise;
  int32_t *path, *n_path, *next;
  int T, V, greedy;   // greedy: every row
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// A logit: NaN reads as -inf, +inf as the largest number.
__device__ __forceinline__ float logit(float x) { return x != x ? -INFINITY : fminf(x, 3.402823466e38f); }

template <typename E>
struct Vec {
  static constexpr int N = 16 / sizeof(E);
};
__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }

// N consecutive elements from i on; `wide`: x + i is 16-byte aligned.
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
__device__ __forceinline__ void logits(const Words<E>& v, float (&y)[Vec<E>::N]) {
#pragma unroll
  for (int j = 0; j < Vec<E>::N; ++j) y[j] = logit(to_float(v.e[j]));
}

// ---------------------------------------------------------------- cluster
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
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

// Every CTA's share of the row's answer. Kinds of values that are reduced, four floats each.
struct Stats {   // maximum and sum of 2^((x - maximum) c), of target and drafter
  float c;
  __device__ __forceinline__ void join(float& m, float& s, float m2, float s2) const {
    const float n = fmaxf(m, m2);
    if (n == -INFINITY) return;   // both empty
    s = (m == n ? s : s * ex2((m - n) * c)) + (m2 == n ? s2 : s2 * ex2((m2 - n) * c));
    m = n;
  }
  __device__ __forceinline__ float4 operator()(float4 a, float4 b) const {
    join(a.x, a.y, b.x, b.y);
    join(a.z, a.w, b.z, b.w);
    return a;
  }
};
struct Sum {
  __device__ __forceinline__ float4 operator()(float4 a, float4 b) const {
    a.x += b.x;
    return a;
  }
};
struct Best {   // the larger value, the lower index where they are equal (y: the index's bits)
  __device__ __forceinline__ float4 operator()(float4 a, float4 b) const {
    const bool take = b.x > a.x || (b.x == a.x && __float_as_int(b.y) < __float_as_int(a.y));
    return take ? b : a;
  }
};

struct Shared {
  float4 warps[kWarps];
  float4 ranks[2][kCluster];   // what each CTA of the cluster found, two calls in turn
  uint64_t kids[FADE_TREE_MAX_NODES + 1];   // children of node i - 1
  // from CTA 0, the same in all: per node its parent, token, uniform number, its target and drafter
  // logits after its parent; then nodes, temperature
  int32_t parent[FADE_TREE_MAX_NODES], token[FADE_TREE_MAX_NODES];
  float u[FADE_TREE_MAX_NODES], tl[FADE_TREE_MAX_NODES], ql[FADE_TREE_MAX_NODES];
  int32_t n;
  float temperature;
  int32_t refused[FADE_TREE_MAX_NODES];
};

// The value over the whole cluster, in every thread; `turn` alternates between calls.
template <class Op>
__device__ __forceinline__ float4 reduce(Shared& sh, float4 v, const Op& op, int& turn) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t rank = cluster_rank(), size = cluster_size();
  auto shuffle = [&](float4 x, int o) {
    return make_float4(__shfl_xor_sync(~0u, x.x, o), __shfl_xor_sync(~0u, x.y, o),
                       __shfl_xor_sync(~0u, x.z, o), __shfl_xor_sync(~0u, x.w, o));
  };
#pragma unroll
  for (int o = 16; o; o >>= 1) v = op(v, shuffle(v, o));
  if (lane == 0) sh.warps[warp] = v;
  __syncthreads();
  if (warp == 0) {
    v = sh.warps[lane & (kWarps - 1)];
#pragma unroll
    for (int o = kWarps / 2; o; o >>= 1) v = op(v, shuffle(v, o));
    if (lane < size) st_remote4(remote(&sh.ranks[turn][rank], lane), v);
  }
  cluster_sync();
  v = sh.ranks[turn][0];
  for (uint32_t r = 1; r < size; ++r) v = op(v, sh.ranks[turn][r]);
  turn ^= 1;
  return v;
}

// The distributions after a node: the vocabulary's logits, and how a thread walks its share.
template <typename E, bool DRAFT>
struct Node {
  static constexpr int N = Vec<E>::N;
  const E *t, *d;
  int V, head, vecs;   // elements before the first 16-byte boundary of t; whole vectors from there
  bool wide_t, wide_d;
  int first, step;     // of this thread's vectors

  // f(index, target logits, drafter logits) for each vector; g the same for single elements, at the ends
  template <class F, class G>
  __device__ __forceinline__ void each(const F& f, const G& g) const {
    for (int v = first; v < vecs; v += kUnroll * step) {
      Words<E> wt[kUnroll], wd[kUnroll];
#pragma unroll
      for (int k = 0; k < kUnroll; ++k) {
        const int at = head + min(v + k * step, vecs - 1) * N;
        load(t, at, true, wt[k]);
        if (DRAFT) load(d, at, wide_d, wd[k]);
      }
#pragma unroll
      for (int k = 0; k < kUnroll; ++k)
        if (v + k * step < vecs) {
          float x[N], y[N];
          logits(wt[k], x);
          if (DRAFT) logits(wd[k], y);
          f(head + (v + k * step) * N, x, y);
        }
    }
    const int ends = V - vecs * N;
    if (first < ends) {
      const int i = first < head ? first : first + vecs * N;
      g(i, logit(to_float(t[i])), DRAFT ? logit(to_float(d[i])) : 0.f);
    }
  }
};

template <typename E, bool DRAFT>
__global__ void __launch_bounds__(kThreads, 4) tree_verify_kernel(const __grid_constant__ Args a) {
  constexpr int N = Vec<E>::N;
  __shared__ Shared sh;
  const int tid = threadIdx.x;
  const uint32_t rank = cluster_rank(), size = cluster_size();
  const int b = blockIdx.x / size;
  int turn = 0;

  auto row_of = [&](int node, const E*& t, const E*& d) {   // logits after a node (-1: the root)
    t = reinterpret_cast<const E*>(node < 0 ? a.target_root + b * a.tr_row
                                            : a.target + b * a.t_row + node * a.t_node);
    d = !DRAFT ? nullptr
               : reinterpret_cast<const E*>(node < 0 ? a.draft_root + b * a.dr_row
                                                     : a.draft + b * a.d_row + node * a.d_node);
  };
  // what CTA 0 reads of the tree is what every CTA decides by
  if (rank == 0) {
    if (tid < a.T) {
      const size_t at = (size_t)b * a.T + tid;
      int parent = a.parents[at];
      if (parent < 0 || parent >= tid) parent = -1;
      const int token = a.tokens[at];
      float tl = -INFINITY, ql = -INFINITY;
      if (token >= 0 && token < a.V && (parent >= 0 || a.target_root)) {
        const E *t, *d;
        row_of(parent, t, d);
        tl = logit(to_float(t[token]));
        if (DRAFT) ql = logit(to_float(d[token]));
      }
      const float u = a.greedy ? 0.f : a.u[at];
      for (uint32_t r = 0; r < size; ++r) {
        st_remote(remote(&sh.parent[tid], r), parent);
        st_remote(remote(&sh.token[tid], r), token);
        st_remote(remote(&sh.u[tid], r), __float_as_uint(u));
        st_remote(remote(&sh.tl[tid], r), __float_as_uint(tl));
        st_remote(remote(&sh.ql[tid], r), __float_as_uint(ql));
      }
    } else if (tid == kThreads - 1) {
      const int n = a.n_nodes ? min(max(a.n_nodes[b], 0), a.T) : a.T;
      const float temp = a.greedy ? 0.f : a.temperature ? a.temperature[b] : 1.f;
      for (uint32_t r = 0; r < size; ++r) {
        st_remote(remote(&sh.n, r), n);
        st_remote(remote(&sh.temperature, r), __float_as_uint(temp));
      }
    }
  }
  if (tid <= FADE_TREE_MAX_NODES) sh.kids[tid] = 0;
  cluster_sync();
  const int n = sh.n;
  if (tid < n)
    atomicOr(reinterpret_cast<unsigned long long*>(&sh.kids[sh.parent[tid] + 1]), 1ull << tid);
  __syncthreads();
  const bool greedy = !(sh.temperature > 0.f);
  const float c = kLog2e / fminf(fmaxf(sh.temperature, 1e-30f), 1e30f);
  const bool lead = rank == 0 && tid == 0;

  int cur = a.target_root ? -1 : 0, kept = 0, next = -1;
  int32_t* path = a.path + (size_t)b * a.T;
  if (!a.target_root && n > 0) {
    if (lead) path[0] = 0;
    kept = 1;
  }
  const bool any = a.target_root || n > 0;   // (no node and no root: nothing to draw from)
  while (any) {
    Node<E, DRAFT> node;
    row_of(cur, node.t, node.d);
    node.V = a.V;
    node.head = min((int)((16 - (reinterpret_cast<uintptr_t>(node.t) & 15)) & 15) / (int)sizeof(E), a.V);
    node.vecs = (a.V - node.head) / N;
    node.wide_d = DRAFT && (reinterpret_cast<uintptr_t>(node.d + node.head) & 15) == 0;
    node.first = rank * kThreads + tid;
    node.step = size * kThreads;
    const uint64_t kids = sh.kids[cur + 1];
    int take = -1;

    if (greedy) {
      float4 best = make_float4(-INFINITY, __int_as_float(0x7fffffff), 0.f, 0.f);
      const Best op;
      auto see = [&](int i, float x) {
        if (x > best.x) best = make_float4(x, __int_as_float(i), 0.f, 0.f);   // ascending in a thread
      };
      node.each(
          [&](int i, const float(&x)[N], const float(&)[N]) {
#pragma unroll
            for (int j = 0; j < N; ++j) see(i + j, x[j]);
          },
          [&](int i, float x, float) {
            best = op(best, make_float4(x, __int_as_float(x == -INFINITY ? 0x7fffffff : i), 0.f, 0.f));
          });
      best = reduce(sh, best, op, turn);
      const int top = best.x == -INFINITY ? -1 : __float_as_int(best.y);
      for (uint64_t left = kids; left && take < 0; left &= left - 1) {
        const int i = __ffsll((long long)left) - 1;
        if (top >= 0 && sh.token[i] == top) take = i;
      }
      next = top;
    } else {
      // -------------------------------------------- maxima and sums
      float4 st = make_float4(-INFINITY, 0.f, -INFINITY, 0.f);
      const Stats join{c};
      auto add = [&](float& m, float& s, const float(&x)[N]) {
        float top = x[0];
#pragma unroll
        for (int j = 1; j < N; ++j) top = fmaxf(top, x[j]);
        if (top > m) {
          s *= ex2((m - top) * c);   // (0 from -inf)
          m = top;
        }
        if (m == -INFINITY) return;
#pragma unroll
        for (int j = 0; j < N; ++j) s += ex2((x[j] - m) * c);
      };
      node.each(
          [&](int, const float(&x)[N], const float(&y)[N]) {
            add(st.x, st.y, x);
            if (DRAFT) add(st.z, st.w, y);
          },
          [&](int, float x, float y) {
            st = join(st, make_float4(x, x == -INFINITY ? 0.f : 1.f, DRAFT ? y : -INFINITY,
                                      DRAFT && y != -INFINITY ? 1.f : 0.f));
          });
      st = reduce(sh, st, join, turn);
      const float mt = st.x == -INFINITY ? 0.f : st.x, md = st.z == -INFINITY ? 0.f : st.z;
      const float it = st.y > 0.f ? 1.f / st.y : 0.f, id = st.w > 0.f ? 1.f / st.w : 0.f;
      // (each product and difference rounded by itself: where p and q are the same numbers, nothing is
      // left of p - q, not what a fused operation would leave)
      auto p_of = [&](float x) { return __fmul_rn(ex2((x - mt) * c), it); };
      auto q_of = [&](float y) { return DRAFT ? __fmul_rn(ex2((y - md) * c), id) : 0.f; };
      float taken = 0.f, left_mass = 1.f;   // a and W
      auto r_of = [&](float p, float q) {
        return DRAFT ? fmaxf(__fsub_rn(p, __fmul_rn(taken, q)), 0.f) : p;
      };

      // -------------------------------------------- children
      int refused = 0;
      for (uint64_t left = kids; left; left &= left - 1) {
        const int i = __ffsll((long long)left) - 1, x = sh.token[i];
        const float p = p_of(sh.tl[i]), q = q_of(sh.ql[i]);
        float r = r_of(p, q);
        if (!DRAFT)
          for (int j = 0; j < refused; ++j)
            if (sh.refused[j] == x) r = 0.f;
        if (sh.u[i] * (DRAFT ? q : 1.f) * left_mass < r) {
          take = i;
          break;
        }
        if (DRAFT) {
          taken += left_mass;
          float4 w = make_float4(0.f, 0.f, 0.f, 0.f);
          auto rest = [&](float x, float y) { w.x += r_of(p_of(x), q_of(y)); };
          node.each(
              [&](int, const float(&x)[N], const float(&y)[N]) {
#pragma unroll
                for (int j = 0; j < N; ++j) rest(x[j], y[j]);
              },
              [&](int, float x, float y) { rest(x, y); });
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
        if (!(left_mass > 0.f)) {   // nothing is left (p and q alike to the last bit): p itself
          taken = 0.f;
          refused = 0;
        }
        float4 best = make_float4(0.f, __int_as_float(0x7fffffff), 0.f, 0.f);
        const Best op;
        const float* noise = a.noise ? a.noise + (size_t)b * a.V : nullptr;
        auto race = [&](int i, float x, float y) {
          float r = r_of(p_of(x), q_of(y));
          if (!DRAFT)
            for (int j = 0; j < refused; ++j)
              if (sh.refused[j] == i) r = 0.f;
          if (r > 0.f) best = op(best, make_float4(noise ? r / noise[i] : r, __int_as_float(i), 0.f, 0.f));
        };
        node.each(
            [&](int i, const float(&x)[N], const float(&y)[N]) {
#pragma unroll
              for (int j = 0; j < N; ++j) race(i + j, x[j], y[j]);
            },
            race);
        best = reduce(sh, best, op, turn);
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
  lc.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim = {kCluster, 1, 1};
  lc.attrs = at;
  lc.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&lc, tree_verify_kernel<E, DRAFT>, a);
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
  const cudaStream_t s = as_stream(stream);
  if (type == FADE_LOGITS_F16) return launch<__half>(a, c->batch, s);
  if (type == FADE_LOGITS_BF16) return launch<__nv_bfloat16>(a, c->batch, s);
  return launch<float>(a, c->batch, s);
}
