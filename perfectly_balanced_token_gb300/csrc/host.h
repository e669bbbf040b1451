// Host side that the C entry points share: argument checks, the plan workspace's
// layout and the launch counter.
#pragma once

#include <algorithm>
#include <atomic>

#include "common.cuh"

namespace moonep {

inline std::atomic<uint64_t> g_launches{0};

inline int check_dims(const moonep_dims* in, Dims* d) {
  if (in == nullptr) return MOONEP_ERR_ARG;
  const moonep_dims& x = *in;
  if (x.R <= 0 || x.E <= 0 || x.K <= 0 || x.S <= 0 || x.H <= 0 || x.Hp <= 0 || x.B < 0)
    return MOONEP_ERR_ARG;
  if (x.mode != 0 && x.mode != 1) return MOONEP_ERR_ARG;
  if (x.policy != 0 && x.policy != 1) return MOONEP_ERR_ARG;
  if (x.gemm_rows != 0 && x.gemm_rows != kMmaM && x.gemm_rows != 2 * kMmaM) return MOONEP_ERR_ARG;
  if (x.E % x.R != 0 || x.K > x.E || x.E > kMaxExperts || x.B > x.E) return MOONEP_ERR_SHAPE;
  if (x.H % 64 != 0 || x.Hp % 64 != 0) return MOONEP_ERR_SHAPE;
  const int64_t N = (int64_t)x.R * x.S * x.K;
  if (N >= (int64_t(1) << 31)) return MOONEP_ERR_SHAPE;
  if ((int64_t)x.R * x.B * x.H >= (int64_t(1) << 31)) return MOONEP_ERR_SHAPE;
  if ((int64_t)x.E * x.H >= (int64_t(1) << 31)) return MOONEP_ERR_SHAPE;
  const int L = x.E / x.R;
  if (x.mode == 0 && x.B < L) return MOONEP_ERR_SLOTS;
  d->R = x.R; d->E = x.E; d->B = x.B; d->K = x.K; d->S = x.S; d->H = x.H; d->Hp = x.Hp;
  d->mode = x.mode;
  d->policy = x.policy;
  d->L = L;
  d->C = x.S * x.K;
  d->N = (int)N;
  d->chunk_tokens = std::max(1, kChunkCopies / x.K);
  d->nchunk = (x.S + d->chunk_tokens - 1) / d->chunk_tokens;
  const int64_t groups = std::min<int64_t>((int64_t)x.E + x.B, d->C);
  d->tile_m = x.gemm_rows;  // 0: the planner chooses per plan
  // room for the longer (128-row) tile list whatever is chosen
  const int64_t mt = (N + kMmaM - 1) / kMmaM + (int64_t)x.R * groups;
  if (mt >= (int64_t(1) << 31)) return MOONEP_ERR_SHAPE;
  d->max_mtiles = (int)mt;
  d->max_groups = (int)std::min<int64_t>((int64_t)x.R * groups, int64_t(1) << 30);
  return MOONEP_OK;
}

inline Layout make_layout(const Dims& d) {
  Layout L{};
  moonep_plan_layout& p = L.pub;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = align256(off + std::max<size_t>(bytes, 4));
    return at;
  };
  p.status = 0;     // status word and counters share the first 256 bytes
  p.counters = 64;
  off = 256;
  const size_t R = d.R, E = d.E, B = d.B, N = d.N, EB = d.E + d.B;
  p.counts = take(4 * R * d.nchunk * E);
  p.T = take(4 * E);
  p.load = take(4 * R);
  p.keep = take(4 * E);
  p.gidx = take(4 * N);
  p.fills = take(4 * 3 * std::max<size_t>(R - 1, 1));
  p.slot_expert = take(4 * R * B);
  p.n_recv = take(4 * R);
  p.src = take(4 * R);
  p.cu_seqlens = take(4 * R * (EB + 1));
  p.dst = take(4 * N);
  p.inverse = take(4 * N);
  p.route = take(4 * N);
  p.pieces = L.pieces = take(sizeof(Piece) * E * R);
  L.piece_n = take(4 * E);
  L.piece_base = take(4 * E * R);
  L.home_base = take(4 * E);
  p.occupied = take(4 * R * B);
  p.reduce = L.red_slots = take(4 * E * R);
  L.red_n = take(4 * E);
  L.red_list = take(4 * E);
  L.rank_tiles = take(4 * (R + 1));
  p.mtiles = take(sizeof(MTile) * (size_t)d.max_mtiles);
  L.rank_groups = take(4 * (R + 1));
  p.groups = take(sizeof(MTile) * (size_t)d.max_groups);
  L.tmaps = take(MOONEP_GEMM_SCRATCH_BYTES);  // last: the layout documents it as the tail
  p.total_bytes = off;
  p.nchunk = d.nchunk;
  p.max_mtiles = d.max_mtiles;
  return L;
}

inline PlanPtrs resolve(const Layout& L, void* ws) {
  char* b = static_cast<char*>(ws);
  const moonep_plan_layout& p = L.pub;
  PlanPtrs q;
  q.status = (int32_t*)(b + p.status);
  q.sched = (int32_t*)(b + p.status + 128);  // inside the 256-byte header the plan zeroes
  q.counters = (int32_t*)(b + p.counters);
  q.counts = (int32_t*)(b + p.counts);
  q.T = (int32_t*)(b + p.T);
  q.load = (int32_t*)(b + p.load);
  q.keep = (int32_t*)(b + p.keep);
  q.gidx = (int32_t*)(b + p.gidx);
  q.fills = (int32_t*)(b + p.fills);
  q.slot_expert = (int32_t*)(b + p.slot_expert);
  q.n_recv = (int32_t*)(b + p.n_recv);
  q.src = (int32_t*)(b + p.src);
  q.cu = (int32_t*)(b + p.cu_seqlens);
  q.dst = (int32_t*)(b + p.dst);
  q.inverse = (int32_t*)(b + p.inverse);
  q.route = (int32_t*)(b + p.route);
  q.pieces = (Piece*)(b + L.pieces);
  q.piece_n = (int32_t*)(b + L.piece_n);
  q.piece_base = (int32_t*)(b + L.piece_base);
  q.home_base = (int32_t*)(b + L.home_base);
  q.occupied = (int32_t*)(b + p.occupied);
  q.red_slots = (int32_t*)(b + L.red_slots);
  q.red_n = (int32_t*)(b + L.red_n);
  q.red_list = (int32_t*)(b + L.red_list);
  q.rank_tiles = (int32_t*)(b + L.rank_tiles);
  q.mtiles = (MTile*)(b + p.mtiles);
  q.rank_groups = (int32_t*)(b + L.rank_groups);
  q.groups = (MTile*)(b + p.groups);
  q.tmaps = (uint8_t*)(((uintptr_t)b + L.tmaps + 127) & ~(uintptr_t)127);
  return q;
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline int finish(cudaError_t e, int launches) {
  g_launches.fetch_add((uint64_t)launches, std::memory_order_relaxed);
  return e == cudaSuccess ? MOONEP_OK : MOONEP_ERR_CUDA;
}

// Common prologue: dims, workspace pointer, alignment of the listed pointers.
#define MOONEP_PROLOGUE(dims, ws)                  \
  Dims d;                                          \
  {                                                \
    const int rc_ = check_dims(dims, &d);          \
    if (rc_ != MOONEP_OK) return rc_;              \
  }                                                \
  if ((ws) == nullptr) return MOONEP_ERR_ARG;      \
  if (!aligned16(ws)) return MOONEP_ERR_ALIGN;     \
  const Layout lay = make_layout(d);               \
  const PlanPtrs P = resolve(lay, const_cast<void*>(static_cast<const void*>(ws)))

#define MOONEP_NEED(ptr)                            \
  do {                                              \
    if ((ptr) == nullptr) return MOONEP_ERR_ARG;    \
    if (!aligned16(ptr)) return MOONEP_ERR_ALIGN;   \
  } while (0)

}  // namespace moonep
