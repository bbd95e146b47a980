// C-ABI host side: handle, argument checks, the window-aware work planner
// (longest-first unit order), workspace, tensor maps and launches.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <mutex>
#include <new>
#include <queue>
#include <vector>

#include <cuda.h>
#include <cuda_runtime.h>

#include "../../include/pa.h"
#include "pa_internal.h"
#include "pa_kv4.h"
#include "pa_pages.h"
#include "pa_ptx.cuh"
#include "pa_qkv.h"
#include "pa_shared.h"

using namespace pa;

namespace {

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  });
  return fn;
}

typedef CUresult (*WriteValue32Fn)(CUstream, CUdeviceptr, cuuint32_t, unsigned int);

// cuStreamWriteValue32: a 32-bit store that a stream performs in order with
// its copies (after a memory barrier), without a kernel
WriteValue32Fn write_value_fn() {
  static WriteValue32Fn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuStreamWriteValue32", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<WriteValue32Fn>(p);
  });
  return fn;
}

struct Plan {
  std::vector<SeqGeom> seqs;
  std::vector<Unit> units;
  std::vector<int> pair_off;  // when the units are assigned to pairs: pair i's first unit (assign_pairs)
  int n_pairs = 0;
  std::vector<Unit> part_units;        // split_units: a unit a part, its place the part's slot
  std::vector<UnitPart> parts;
  std::vector<SplitUnit> split;
  int n_stored_blocks = 0;
  int n_tok_total = 0;
  int total_q = 0;
  long long n_tiles = 0;
};

// Host planner: per-sequence widened geometry and the work units sorted by
// decreasing cost (tiles), so the longest units start first.
int build_plan(int HQ, int HKV, int n_seq, const pa_seq* seqs, int S, int W, int max_pages, Plan& P) {
  if (HQ <= 0 || HKV <= 0 || HQ % HKV != 0) return PA_EINVAL;
  const int G = HQ / HKV;
  if (G > kRows || kRows % G != 0) return PA_EINVAL;
  if (n_seq <= 0 || seqs == nullptr || S < 0) return PA_EINVAL;
  const int UT = kUnitRows / G;  // tokens per unit
  P = Plan();
  int tok_off = 0;
  for (int s = 0; s < n_seq; ++s) {
    const pa_seq& q = seqs[s];
    if (q.n_q < 1 || q.q_start < 0 || q.q_off < 0 || q.n_ctx < q.q_start + q.n_q) return PA_EINVAL;
    if (max_pages > 0 && (long long)q.n_ctx > (long long)max_pages * kPage) return PA_EINVAL;
    if ((long long)q.q_off + q.n_q > (1LL << 30) || (long long)q.n_ctx > (1LL << 30)) return PA_EINVAL;
    SeqGeom g{};
    g.q_off = q.q_off;
    g.q_start = q.q_start;
    g.n_q = q.n_q;
    g.n_ctx = q.n_ctx;
    g.tok_off = tok_off;
    g.bt_row = s;
    seq_geom_fill(g, S, W);
    tok_off += g.n_blocks * kPage;
    if (tok_off > (1 << 30)) return PA_EINVAL;
    P.seqs.push_back(g);
    P.total_q = std::max(P.total_q, q.q_off + q.n_q);
    const int t_first = (q.q_start / UT) * UT;
    for (int t0 = t_first; t0 < q.q_start + q.n_q; t0 += UT) {
      const UnitGeom ug = unit_geom(t0, UT, g, S, W);
      for (int kv = 0; kv < HKV; ++kv) {
        P.units.push_back(Unit{s, kv, t0, ug.n_tiles});
        P.n_tiles += ug.n_tiles;
      }
    }
  }
  std::stable_sort(P.units.begin(), P.units.end(), [](const Unit& a, const Unit& b) { return a.n_tiles > b.n_tiles; });
  P.n_stored_blocks = tok_off / kPage;
  P.n_tok_total = tok_off;
  return PA_OK;
}

// A pair's change of unit costs about two tiles' time (the unit's last PV and
// the epilogue, the next unit's Q rows and first QK^T; clock64 stamps on
// GB300), so a unit weighs its tiles plus that.
constexpr int kUnitSwitchTiles = 2;
// The attention kernel's pairs for n units: one per co-resident cluster slot,
// at most one per unit.
int launch_pairs(int n_sm, int n) { return std::max(1, std::min(n, pa::attention_pairs(n_sm))); }
// Unit records (16 bytes) that hold n_pairs + 1 pair offsets after a unit list.
size_t pair_off_records(int n_pairs) { return ((size_t)n_pairs + 1 + 3) / 4; }
// Units sorted longest first, assigned to n_pairs SM pairs: each to the pair
// whose work so far is least (ties: the lowest pair), a greedy
// longest-first schedule; then laid out pair by pair, each pair's units still
// longest first.  off[i] = pair i's first unit, off[n_pairs] = n.  Against
// walking the sorted list with stride n_pairs (pair i: units i, i + n_pairs,
// ...), the most loaded pair's work falls from 1.28x the mean to 1.04x at 4k
// tokens (256 units), 1.09x to 1.01x for the chunked batch, 1.02x to 1.00x at
// 32k.
void assign_pairs(const Unit* units, int n, int n_pairs, std::vector<Unit>& out, std::vector<int>& off) {
  using Load = std::pair<long long, int>;  // (work so far, pair)
  std::priority_queue<Load, std::vector<Load>, std::greater<Load>> q;
  for (int i = 0; i < n_pairs; ++i) q.push(Load{0, i});
  std::vector<int> pair_of((size_t)n);
  std::vector<int> count((size_t)n_pairs, 0);
  for (int u = 0; u < n; ++u) {
    const Load top = q.top();
    q.pop();
    pair_of[(size_t)u] = top.second;
    ++count[(size_t)top.second];
    q.push(Load{top.first + units[u].n_tiles + kUnitSwitchTiles, top.second});
  }
  off.assign((size_t)n_pairs + 1, 0);
  for (int i = 0; i < n_pairs; ++i) off[(size_t)i + 1] = off[(size_t)i] + count[(size_t)i];
  out.resize((size_t)n);
  std::vector<int> next(off.begin(), off.end() - 1);
  for (int u = 0; u < n; ++u) out[(size_t)next[(size_t)pair_of[(size_t)u]]++] = units[u];
}

// The units of a call of fewer than n_pairs units with their keys split, so that the longest part has as few tiles as
// one part a pair allows; none where that saves too little.  A tile takes about 1.4 us; a third launch costs two or
// three of them, the partials, written and read back, one more for every 24 parts or so.  GB300, 16 query and 2 kv heads,
// us a call whole and split: 30 tokens behind 256 (1 tile saved, 4 parts) 15.1 and 16.7, behind 380 (2) 16.7 and 17.3, behind
// 500 (3) 18.1 and 17.3, behind 640 (4) 19.7 and 17.4, behind 3000 47.0 and 21.1, behind 16000 193 and 33.4; 8 sequences of
// 30 behind 1000 (4 saved, 64 parts) 27.0 and 28.0, behind 1200 (5) 30.7 and 29.9, behind 2000 41.6 and 37.0; 800 tokens
// behind 1000 (3 saved, parts for all pairs) 32.5 and 40.2.  Parts of at least two tiles: 30 tokens behind 2000 took 23.3
// (before the launches overlapped), with one tile at least 26.7, with three 25.1, with four 25.4.
constexpr int kSplitLeast = 2;
constexpr int split_cost(long long parts) { return 3 + (int)(parts / 24); }
void split_units(Plan& P, int n_pairs) {
  const int n = (int)P.units.size();
  if (n >= n_pairs) return;
  const int most = P.units[0].n_tiles;  // longest first
  int lo = kSplitLeast, hi = std::max(lo, most);
  const auto count = [&](int T) {
    long long c = 0;
    for (const Unit& u : P.units) c += (u.n_tiles + T - 1) / T;
    return c;
  };
  while (lo < hi) {
    const int mid = (lo + hi) / 2;
    if (count(mid) <= n_pairs) hi = mid;
    else lo = mid + 1;
  }
  if (count(lo) > n_pairs || most - lo < split_cost(count(lo))) return;
  for (const Unit& u : P.units) {
    const int k = (u.n_tiles + lo - 1) / lo;
    P.split.push_back(SplitUnit{u.seq, u.g, u.t0, (int)P.parts.size(), k, {0, 0, 0}});
    for (int i = 0; i < k; ++i) {
      const int a = (int)((long long)i * u.n_tiles / k), b = (int)((long long)(i + 1) * u.n_tiles / k);
      P.parts.push_back(UnitPart{a, b - a});
      P.part_units.push_back(Unit{u.seq, u.g, u.t0, b - a});
    }
  }
}

bool same_plan_key(const std::vector<int>& a, const std::vector<int>& b) { return a == b; }

// The host-buffer path's chunks: ends (rows of the sequences laid end to end)
// of chunks of work units counted in waves (a wave: one unit for every one of
// the n_pairs SM pairs the kernel runs at once; a part-filled wave leaves
// pairs idle): one wave first and one wave last, two in between.  The short
// first chunk starts the computation and the copy-out early, the short last
// one shortens what is left after the last rows are in; two waves between
// keep the launches few (at 32k tokens on GB300: 921 TOPS end to end against
// 888 with two-wave chunks throughout, 896-904 with three-wave middles or
// half-wave ends).  A boundary inside a sequence moves to a multiple of a
// unit's tokens (down, or up to the sequence's end when that would empty the
// piece), so every unit lies in one chunk.  ends is increasing, last = total rows.
int host_chunk_ends(int HQ, int HKV, int n_seq, const pa_seq* seqs, int n_pairs, std::vector<long long>& ends) {
  if (HQ <= 0 || HKV <= 0 || HQ % HKV != 0 || kUnitRows % (HQ / HKV) != 0) return PA_EINVAL;
  if (n_seq <= 0 || seqs == nullptr || n_pairs <= 0) return PA_EINVAL;
  std::vector<long long> base(n_seq + 1, 0);  // first row of each sequence, end to end
  for (int s = 0; s < n_seq; ++s) {
    if (seqs[s].n_q < 1 || seqs[s].q_start < 0) return PA_EINVAL;
    base[s + 1] = base[s] + seqs[s].n_q;
  }
  const long long T = base[n_seq];
  const long long UT = kUnitRows / (HQ / HKV);  // tokens per unit
  const long long wave = std::max(UT, (long long)n_pairs * UT / HKV);
  std::vector<long long> cuts;
  for (long long at = 0; at < T;) {
    long long step = at == 0 ? wave : 2 * wave;
    if (T - at > wave && T - at - step < wave) step = T - at - wave;  // a last chunk of one wave
    at = std::min(T, at + step);
    cuts.push_back(at);
  }
  ends.clear();
  for (long long cut : cuts) {
    const int s = (int)(std::upper_bound(base.begin(), base.end(), cut) - base.begin()) - 1;
    if (s >= 0 && s < n_seq && cut != base[s]) {  // inside sequence s
      const long long abs_pos = seqs[s].q_start + (cut - base[s]);
      long long r = abs_pos / UT * UT;
      if (r <= seqs[s].q_start) r = std::min((long long)seqs[s].q_start + seqs[s].n_q, (abs_pos / UT + 1) * UT);
      cut = base[s] + (r - seqs[s].q_start);
    }
    if (ends.empty() || cut > ends.back()) ends.push_back(cut);
  }
  return PA_OK;
}

}  // namespace

// A device buffer that grows; the ones it outgrew are freed with the handle.
struct Workspace {
  void* p = nullptr;
  size_t bytes = 0;
  std::vector<void*> outgrown;
};

struct pa_ctx {
  int HQ = 0, HKV = 0, G = 0, TQ = 0, n_pool = 0, max_pages = 0;
  pa_options opt{};
  int device = 0, n_sm = 0;

  // workspace
  __nv_bfloat16* kw = nullptr;
  __half* vt = nullptr;
  float* ks = nullptr;
  float* vs = nullptr;
  int n_tok_cap = 0;
  unsigned int* vsmax = nullptr;
  int vsmax_cap = 0;
  SeqGeom* d_seqs = nullptr;
  int seqs_cap = 0;
  Unit* d_units = nullptr;
  int units_cap = 0;
  int* d_err = nullptr;  // kErrWords
  unsigned int* d_qflags = nullptr;  // host path: chunk c's q rows are in when d_qflags[c] == q_epoch
  int qflags_cap = 0;
  unsigned int q_epoch = 0;

  // plan upload through pinned staging
  void* h_stage = nullptr;
  size_t h_stage_cap = 0;
  cudaEvent_t upload_done = nullptr;
  bool upload_recorded = false;
  std::vector<int> plan_key;
  Plan plan;

  // tensor maps
  AttnMaps maps{};
  const void* kv_ptr = nullptr;
  int kv_rows = -1;
  int kv_cap = -1;

  // decode: partials, the pairs' tickets (zeroed once; the kernel leaves them
  // at zero), the pool's tensor maps (cached by pool pointers)
  DecodeMaps dec_maps{};
  const void* dec_kp = nullptr;
  const void* dec_vp = nullptr;
  float* d_part = nullptr;
  int part_cap = 0;
  unsigned long long* d_tickets = nullptr;
  int tickets_cap = 0;

  // shared-prefix decode: partials of the prefix and of the sequences' own keys.  A buffer that became too
  // small is kept until the handle goes, since a captured graph may still write it.
  Workspace sh_pre, sh_own;
  // 4-bit decode: partials (as above); compaction: marks, moves
  Workspace k4_part, pages;
  Workspace att_part;  // 4-bit prefill: partials of split units
  int sh_pass = -1;  // pa_debug_decode_shared_pass

  // host-buffer path staging
  void* hb[7] = {nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr};
  size_t hb_cap[7] = {0, 0, 0, 0, 0, 0, 0};
  cudaStream_t s_h2d = nullptr, s_d2h = nullptr;  // the host path's copy streams
  std::vector<cudaEvent_t> pipe_ev;                // and its events (no timing)
  SeqGeom* d_pseqs = nullptr;                      // its chunks' plans, uploaded together
  int pseqs_cap = 0;
  Unit* d_punits = nullptr;
  int punits_cap = 0;
  void* h_pstage = nullptr;
  size_t h_pstage_cap = 0;
  cudaEvent_t pstage_done = nullptr;
  bool pstage_recorded = false;

  // timing
  std::vector<cudaEvent_t> ev_free;
  std::vector<cudaEvent_t> ev_pending;  // triples (before widen, after widen, after attention)
  double t_widen = 0.0, t_attn = 0.0;
  int t_calls = 0;
};

namespace {

int cuda_fail(cudaError_t e) {
  (void)cudaGetLastError();  // reported once: not to be found again behind the next launch
  if (e == cudaErrorMemoryAllocation) return PA_ENOMEM;
  return PA_ECUDA;
}

#define PA_CUDA(x)                              \
  do {                                          \
    cudaError_t e_ = (x);                       \
    if (e_ != cudaSuccess) return cuda_fail(e_); \
  } while (0)

template <typename T>
int grow(T*& p, int& cap, size_t need) {
  if ((size_t)cap >= need) return PA_OK;
  size_t n = std::max(need, (size_t)cap + (size_t)cap / 2);
  if (p) PA_CUDA(cudaFree(p));
  p = nullptr;
  cap = 0;
  PA_CUDA(cudaMalloc(reinterpret_cast<void**>(&p), n * sizeof(T)));
  cap = (int)n;
  return PA_OK;
}

int grow_bytes(void*& p, size_t& cap, size_t need) {
  if (cap >= need) return PA_OK;
  size_t n = std::max(need, cap + cap / 2);
  if (p) PA_CUDA(cudaFree(p));
  p = nullptr;
  cap = 0;
  PA_CUDA(cudaMalloc(&p, n));
  cap = n;
  return PA_OK;
}

int reserve(Workspace& w, size_t need, bool capturing) {
  if (w.bytes >= need) return PA_OK;
  if (capturing) return PA_ENOMEM;  // an allocation would end the capture
  const size_t n = std::max(need, w.bytes + w.bytes / 2);
  void* p = nullptr;
  PA_CUDA(cudaMalloc(&p, n));
  if (w.p) w.outgrown.push_back(w.p);
  w.p = p;
  w.bytes = n;
  return PA_OK;
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// A decode launch's CTA runs: first block, its sequence, the CTA's partial slot in its pair.
struct DecRuns {
  std::vector<int> x0, seq, slot;
  int max_slots = 1;
};

int encode(CUtensorMap* m, CUtensorMapDataType dt, int rank, const void* base, const uint64_t* dims,
           const uint64_t* strides_bytes, const uint32_t* box, CUtensorMapSwizzle sw) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return PA_ECUDA;
  cuuint64_t d[5], s[4];
  cuuint32_t b[5], es[5];
  for (int i = 0; i < rank; ++i) {
    d[i] = dims[i];
    b[i] = box[i];
    es[i] = 1;
  }
  for (int i = 0; i < rank - 1; ++i) s[i] = strides_bytes[i];
  CUresult r = fn(m, dt, (cuuint32_t)rank, const_cast<void*>(base), d, s, b, es, CU_TENSOR_MAP_INTERLEAVE_NONE, sw,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? PA_OK : PA_ECUDA;
}

// The split units as records after a unit list: SplitUnit, Unit, UnitPart arrays.
static_assert(sizeof(SplitUnit) == 2 * sizeof(Unit) && sizeof(Unit) == 2 * sizeof(UnitPart) && sizeof(Unit) == 16, "records");
size_t split_records(const Plan& P) { return 2 * P.split.size() + P.part_units.size() + (P.parts.size() + 1) / 2; }
void stage_split(const Plan& P, char* to) {
  if (P.split.empty()) return;
  std::memcpy(to, P.split.data(), P.split.size() * sizeof(SplitUnit));
  to += P.split.size() * sizeof(SplitUnit);
  std::memcpy(to, P.part_units.data(), P.part_units.size() * sizeof(Unit));
  std::memcpy(to + P.part_units.size() * sizeof(Unit), P.parts.data(), P.parts.size() * sizeof(UnitPart));
}

// Plan (cached by its inputs), workspace sizing and the upload of the plan.
// Widened-row workspace for at least `rows` rows (reallocating frees the old
// buffers, which waits for the device).
int reserve_rows(pa_handle h, size_t rows) {
  const size_t need_tok = (rows + 63) / 64 * 64;
  if ((size_t)h->n_tok_cap >= need_tok) return PA_OK;
  size_t cap = std::max(need_tok, (size_t)h->n_tok_cap + (size_t)h->n_tok_cap / 2);
  cap = (cap + 63) / 64 * 64;
  if (h->kw) cudaFree(h->kw);
  if (h->vt) cudaFree(h->vt);
  if (h->ks) cudaFree(h->ks);
  if (h->vs) cudaFree(h->vs);
  h->kw = nullptr;
  h->vt = nullptr;
  h->ks = nullptr;
  h->vs = nullptr;
  h->n_tok_cap = 0;
  h->kv_ptr = nullptr;
  PA_CUDA(cudaMalloc(&h->kw, cap * h->HKV * kHeadDim * sizeof(__nv_bfloat16)));
  PA_CUDA(cudaMalloc(&h->vt, cap * h->HKV * kHeadDim * sizeof(__half)));
  PA_CUDA(cudaMalloc(&h->ks, cap * h->HKV * sizeof(float)));
  PA_CUDA(cudaMalloc(&h->vs, cap * h->HKV * sizeof(float)));
  h->n_tok_cap = (int)cap;
  return PA_OK;
}

int prepare(pa_handle h, int n_seq, const pa_seq* seqs, int S, int W, cudaStream_t st, bool split = false) {
  std::vector<int> key;
  key.reserve(4 + 4 * n_seq);
  key.push_back(split);
  key.push_back(n_seq);
  key.push_back(S);
  key.push_back(W);
  for (int s = 0; s < n_seq; ++s) {
    key.push_back(seqs[s].q_off);
    key.push_back(seqs[s].q_start);
    key.push_back(seqs[s].n_q);
    key.push_back(seqs[s].n_ctx);
  }
  int rc;
  if (!h->plan_key.empty() && same_plan_key(key, h->plan_key)) {
    // another call may have lost the workspace since, in an allocation that failed
    if ((rc = reserve_rows(h, (size_t)h->plan.n_tok_total))) return rc;
    return grow(h->vsmax, h->vsmax_cap, 2 * (size_t)n_seq * h->HKV);
  }
  Plan P;
  rc = build_plan(h->HQ, h->HKV, n_seq, seqs, S, W, h->max_pages, P);
  if (rc) return rc;
  // the units laid out pair by pair for the kernel's pairs, the pair offsets after them
  const int n_u = (int)P.units.size();
  P.n_pairs = launch_pairs(h->n_sm, n_u);
  if (split && h->opt.p_mode == PA_P_F16) split_units(P, attention_pairs(h->n_sm));
  {
    std::vector<Unit> by_pair;
    assign_pairs(P.units.data(), n_u, P.n_pairs, by_pair, P.pair_off);
    P.units = std::move(by_pair);
  }
  // and the split units after those
  const size_t n_whole = (size_t)n_u + pair_off_records(P.n_pairs);
  const size_t n_rec = n_whole + split_records(P);
  h->plan_key.clear();  // from here on the tables on the device may be another plan's than h->plan, or gone
  // workspace
  if ((rc = reserve_rows(h, (size_t)P.n_tok_total))) return rc;
  if ((rc = grow(h->vsmax, h->vsmax_cap, 2 * (size_t)n_seq * h->HKV))) return rc;
  if ((rc = grow(h->d_seqs, h->seqs_cap, P.seqs.size()))) return rc;
  if ((rc = grow(h->d_units, h->units_cap, n_rec))) return rc;
  // upload through pinned staging; never overwrite staging a copy may still read
  const size_t bytes_s = P.seqs.size() * sizeof(SeqGeom), bytes_u = n_rec * sizeof(Unit);
  if (h->upload_recorded) PA_CUDA(cudaEventSynchronize(h->upload_done));
  if (h->h_stage_cap < bytes_s + bytes_u) {
    if (h->h_stage) cudaFreeHost(h->h_stage);
    h->h_stage = nullptr;
    h->h_stage_cap = 0;
    PA_CUDA(cudaMallocHost(&h->h_stage, bytes_s + bytes_u));
    h->h_stage_cap = bytes_s + bytes_u;
  }
  std::memcpy(h->h_stage, P.seqs.data(), bytes_s);
  std::memcpy(static_cast<char*>(h->h_stage) + bytes_s, P.units.data(), (size_t)n_u * sizeof(Unit));
  std::memcpy(static_cast<char*>(h->h_stage) + bytes_s + (size_t)n_u * sizeof(Unit), P.pair_off.data(),
              P.pair_off.size() * sizeof(int));
  stage_split(P, static_cast<char*>(h->h_stage) + bytes_s + n_whole * sizeof(Unit));
  PA_CUDA(cudaMemcpyAsync(h->d_seqs, h->h_stage, bytes_s, cudaMemcpyHostToDevice, st));
  PA_CUDA(cudaMemcpyAsync(h->d_units, static_cast<char*>(h->h_stage) + bytes_s, bytes_u, cudaMemcpyHostToDevice, st));
  PA_CUDA(cudaEventRecord(h->upload_done, st));
  h->upload_recorded = true;
  h->plan = std::move(P);
  h->plan_key = std::move(key);
  return PA_OK;
}

int check_inputs(pa_handle h, const void* q, const int8_t* kp, const int8_t* vp, const float* ksc, const float* vsc,
                 const int32_t* bt, const void* out) {
  if (!h) return PA_EINVAL;
  if (!q || !kp || !vp || !ksc || !vsc || !bt || !out) return PA_EINVAL;
  if (!aligned(q, 16) || !aligned(kp, 16) || !aligned(vp, 16) || !aligned(out, 16)) return PA_EINVAL;
  if (!aligned(ksc, 4) || !aligned(vsc, 4) || !aligned(bt, 4)) return PA_EINVAL;
  return PA_OK;
}

WidenParams widen_params(pa_handle h, const int8_t* kp, const int8_t* vp, const float* ksc, const float* vsc,
                         const int32_t* bt, int n_seq, const SeqGeom* d_seqs = nullptr, int n_stored_blocks = -1) {
  WidenParams w{};
  w.k_pool = kp;
  w.v_pool = vp;
  w.k_scale = ksc;
  w.v_scale = vsc;
  w.block_table = bt;
  w.bt_stride = h->max_pages;
  w.n_pool = h->n_pool;
  w.HKV = h->HKV;
  w.seqs = d_seqs ? d_seqs : h->d_seqs;
  w.n_seq = n_seq;
  w.n_stored_blocks = n_stored_blocks >= 0 ? n_stored_blocks : h->plan.n_stored_blocks;
  w.n_tok_cap = h->n_tok_cap;
  w.kw = h->kw;
  w.vt = h->vt;
  w.ks = h->ks;
  w.vs = h->vs;
  w.vsmax = h->vsmax;
  w.err = h->d_err;
  return w;
}

cudaEvent_t take_event(pa_handle h) {
  if (!h->ev_free.empty()) {
    cudaEvent_t e = h->ev_free.back();
    h->ev_free.pop_back();
    return e;
  }
  cudaEvent_t e = nullptr;
  if (cudaEventCreate(&e) != cudaSuccess) return nullptr;
  return e;
}

// The widening pass of plan P, whose sequence table is already on the device
// at d_seqs (the caller has sized the widened workspace for P).
int launch_widen_plan(pa_handle h, const Plan& P, const SeqGeom* d_seqs, int n_seq, const int8_t* kp,
                      const int8_t* vp, const float* ksc, const float* vsc, const int32_t* bt, float sm_scale,
                      cudaStream_t st, const uint8_t* pool4 = nullptr) {
  if (!pool4) PA_CUDA(cudaMemsetAsync(h->vsmax, 0, sizeof(unsigned int) * n_seq * h->HKV, st));
  WidenParams wp = widen_params(h, kp, vp, ksc, vsc, bt, n_seq, d_seqs, P.n_stored_blocks);
  wp.k_mult = sm_scale * 1.4426950408889634f;  // the softmax's sm_scale * log2(e), folded into the K scales
  PA_CUDA(pool4 ? launch_widen_kv4(wp, pool4, st) : launch_widen(wp, st));
  return PA_OK;
}

// The attention kernel over n_units work units at d_units, all of plan P
// (whose sequence table is on the device at d_seqs and whose pages the
// widening pass has already written).
int launch_attention_plan(pa_handle h, const Plan& P, const SeqGeom* d_seqs, const Unit* d_units, int n_units,
                          const void* q, int S, int W, float sm_scale, void* out, cudaStream_t st,
                          const void* gate, bool overlap_prev = false, const unsigned int* q_ready = nullptr,
                          unsigned int q_epoch = 0, const int* d_pair_off = nullptr, int plan_pairs = 0,
                          bool kv4 = false, const AttnSplit* split = nullptr, const SplitUnit* split_units = nullptr) {
  int rc = PA_OK;
  // tensor maps
  if (h->kw != h->kv_ptr || P.n_tok_total != h->kv_rows || h->n_tok_cap != h->kv_cap) {
    const uint64_t kd[3] = {(uint64_t)kHeadDim, (uint64_t)P.n_tok_total, (uint64_t)h->HKV};
    const uint64_t kst[2] = {(uint64_t)kHeadDim * 2, (uint64_t)h->n_tok_cap * kHeadDim * 2};
    const uint32_t kbox[3] = {64, (uint32_t)kTileKeys / 2, 1};  // one CTA's half of a tile
    if ((rc = encode(&h->maps.k, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, h->kw, kd, kst, kbox,
                     CU_TENSOR_MAP_SWIZZLE_128B)))
      return rc;
    const uint64_t vd[3] = {(uint64_t)P.n_tok_total, (uint64_t)kHeadDim, (uint64_t)h->HKV};
    const uint64_t vst[2] = {(uint64_t)h->n_tok_cap * 2, (uint64_t)h->n_tok_cap * kHeadDim * 2};
    const uint32_t vbox[3] = {(uint32_t)kChunkKeys, (uint32_t)kHeadDim / 2, 1};  // one CTA's half of the dims
    if ((rc = encode(&h->maps.v, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, h->vt, vd, vst, vbox,
                     CU_TENSOR_MAP_SWIZZLE_128B)))
      return rc;
    h->kv_ptr = h->kw;
    h->kv_rows = P.n_tok_total;
    h->kv_cap = h->n_tok_cap;
  }
  // the query's map: q as [tokens][HQ][256], a unit's rows are TQ tokens x G heads
  AttnMaps maps = h->maps;
  {
    const uint64_t qd[3] = {(uint64_t)kHeadDim, (uint64_t)h->HQ, (uint64_t)P.total_q};
    const uint64_t qst[2] = {(uint64_t)kHeadDim * 2, (uint64_t)h->HQ * kHeadDim * 2};
    const uint32_t qbox[3] = {64, (uint32_t)h->G, (uint32_t)h->TQ};
    if ((rc = encode(&maps.q, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, q, qd, qst, qbox, CU_TENSOR_MAP_SWIZZLE_128B)))
      return rc;
  }
  AttnParams a{};
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.total_q = P.total_q;
  a.seqs = d_seqs;
  a.units = d_units;
  a.n_units = n_units;
  a.pair_off = d_pair_off;
  a.plan_pairs = plan_pairs;
  a.ks = h->ks;
  a.vs = h->vs;
  a.vsmax = h->vsmax;
  a.out = static_cast<__nv_bfloat16*>(out);
  a.gate = static_cast<const __nv_bfloat16*>(gate);
  a.HQ = h->HQ;
  a.HKV = h->HKV;
  a.G = h->G;
  a.TQ = h->TQ;
  a.n_tok_cap = h->n_tok_cap;
  a.S = S;
  a.W = W;
  a.sm_scale_log2 = sm_scale * 1.4426950408889634f;
  a.q_mode = h->opt.q_mode;
  a.p_mode = h->opt.p_mode;
  a.err = h->d_err;
  a.wait_ns = (unsigned long long)h->opt.wait_timeout_ms * 1000000ull;
  a.q_ready = q_ready;
  a.q_epoch = q_epoch;
  a.debug_stall = h->opt.debug_stall;
  a.kv4 = kv4;
  a.n_seq = (int)P.seqs.size();
  if (split) PA_CUDA(launch_attention_split(a, maps, *split, split_units, (int)P.split.size(), st));
  else PA_CUDA(launch_attention(a, maps, h->n_sm, st, overlap_prev));
  return PA_OK;
}

// Events for pa_timing around a widening pass and the attention work after
// it: mark(0) before the pass, mark(1) after it, mark(2) after the attention.
struct TimingMarks {
  cudaEvent_t e[3] = {nullptr, nullptr, nullptr};
  bool queued = false;  // mark(2) handed the events to the pending list
  // events of a call that failed before its last mark go back to the free list
  void release(pa_handle h) {
    if (queued) return;
    for (auto& x : e)
      if (x) h->ev_free.push_back(x);
    e[0] = e[1] = e[2] = nullptr;
  }
  int init(pa_handle h) {
    if (!h->opt.record_timing) return PA_OK;
    for (auto& x : e)
      if (!(x = take_event(h))) return PA_ECUDA;
    return PA_OK;
  }
  int mark(pa_handle h, int i, cudaStream_t st) {
    if (!e[i]) return PA_OK;
    PA_CUDA(cudaEventRecord(e[i], st));
    if (i == 2) {
      for (auto& x : e) h->ev_pending.push_back(x);
      queued = true;
    }
    return PA_OK;
  }
};

// The widening pass and the attention kernel of plan P, whose sequence table
// and unit list are already on the device at d_seqs / d_units (the caller
// has sized the widened workspace for P).
int launch_plan(pa_handle h, const Plan& P, const SeqGeom* d_seqs, const Unit* d_units, int n_seq, const void* q,
                const int8_t* kp, const int8_t* vp, const float* ksc, const float* vsc, const int32_t* bt, int S,
                int W, float sm_scale, void* out, cudaStream_t st, const void* gate, const uint8_t* pool4 = nullptr) {
  TimingMarks tm;
  int rc;
  if (!P.split.empty()) {  // few units on the 4-bit pool (the int8 pool's calls keep their units whole)
    const size_t rows = P.parts.size() * (size_t)kUnitRows, o_bytes = rows * kHeadDim * sizeof(float);
    if ((rc = reserve(h->att_part, o_bytes + rows * sizeof(float2), false))) return rc;
    const Unit* rec = d_units + P.units.size() + pair_off_records(P.n_pairs);
    const SplitUnit* su = reinterpret_cast<const SplitUnit*>(rec);
    const Unit* pu = rec + 2 * P.split.size();
    AttnSplit sp{reinterpret_cast<const UnitPart*>(pu + P.part_units.size()), static_cast<float*>(h->att_part.p),
                 reinterpret_cast<float2*>(static_cast<char*>(h->att_part.p) + o_bytes)};
    if (!(rc = tm.init(h)) && !(rc = tm.mark(h, 0, st)) &&
        !(rc = launch_widen_plan(h, P, d_seqs, n_seq, kp, vp, ksc, vsc, bt, sm_scale, st, pool4)) &&
        !(rc = tm.mark(h, 1, st)) &&
        !(rc = launch_attention_plan(h, P, d_seqs, pu, (int)P.part_units.size(), q, S, W, sm_scale, out, st, gate, false,
                                     nullptr, 0, nullptr, 0, true, &sp, su)))
      rc = tm.mark(h, 2, st);
    if (rc) tm.release(h);
    return rc;
  }
  if (!(rc = tm.init(h)) && !(rc = tm.mark(h, 0, st)) &&
      !(rc = launch_widen_plan(h, P, d_seqs, n_seq, kp, vp, ksc, vsc, bt, sm_scale, st, pool4)) &&
      !(rc = tm.mark(h, 1, st)) &&
      !(rc = launch_attention_plan(h, P, d_seqs, d_units, (int)P.units.size(), q, S, W, sm_scale, out, st, gate,
                                   false, nullptr, 0, reinterpret_cast<const int*>(d_units + P.units.size()),
                                   P.n_pairs, pool4 != nullptr)))
    rc = tm.mark(h, 2, st);
  if (rc) tm.release(h);
  return rc;
}

int run(pa_handle h, int n_seq, const pa_seq* seqs, const void* q, const int8_t* kp, const int8_t* vp,
        const float* ksc, const float* vsc, const int32_t* bt, int S, int W, float sm_scale, void* out,
        cudaStream_t st, const void* gate = nullptr) {
  int rc = check_inputs(h, q, kp, vp, ksc, vsc, bt, out);
  if (rc) return rc;
  if (gate && !aligned(gate, 16)) return PA_EINVAL;
  if (!(sm_scale == sm_scale) || sm_scale < 0.f) return PA_EINVAL;
  if ((rc = prepare(h, n_seq, seqs, S, W, st))) return rc;
  return launch_plan(h, h->plan, h->d_seqs, h->d_units, n_seq, q, kp, vp, ksc, vsc, bt, S, W, sm_scale, out, st,
                     gate);
}

}  // namespace

extern "C" {

void pa_default_options(pa_options* opt) {
  if (!opt) return;
  opt->q_mode = PA_Q_BF16;
  opt->p_mode = PA_P_F16;
  opt->wait_timeout_ms = 2000;
  opt->record_timing = 0;
  opt->debug_stall = 0;
  opt->debug_fail_host = 0;
}

const char* pa_strerror(int code) {
  switch (code) {
    case PA_OK: return "ok";
    case PA_EINVAL: return "invalid argument";
    case PA_EARCH: return "device is not an sm_103 GPU";
    case PA_ECUDA: return "CUDA call failed";
    case PA_ETIMEOUT: return "device-side wait timed out";
    case PA_EBADPAGE: return "block-table entry outside the pool";
    case PA_ENOMEM: return "out of device memory";
    case PA_ENOSCRATCH: return "call exceeds the static scratch of pa_prefill_noalloc";
    default: return "unknown error";
  }
}

int pa_create(pa_handle* out, int n_q_heads, int n_kv_heads, int head_dim, int page_size, int n_pool_pages,
              int max_pages_per_seq, const pa_options* opt) {
  if (!out) return PA_EINVAL;
  *out = nullptr;
  if (head_dim != kHeadDim || page_size != kPage) return PA_EINVAL;
  if (n_q_heads <= 0 || n_kv_heads <= 0 || n_kv_heads > 8 || n_q_heads % n_kv_heads) return PA_EINVAL;
  const int G = n_q_heads / n_kv_heads;
  if (G > kRows || kRows % G) return PA_EINVAL;
  if (n_pool_pages <= 0 || max_pages_per_seq <= 0) return PA_EINVAL;
  pa_options o;
  pa_default_options(&o);
  if (opt) o = *opt;
  if ((o.q_mode != PA_Q_BF16 && o.q_mode != PA_Q_INT8) || (o.p_mode != PA_P_F16 && o.p_mode != PA_P_U8) ||
      o.wait_timeout_ms <= 0)
    return PA_EINVAL;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return PA_ECUDA;
  cudaDeviceProp prop;
  if (cudaGetDeviceProperties(&prop, dev) != cudaSuccess) return PA_ECUDA;
  if (prop.major != 10 || prop.minor != 3) return PA_EARCH;
  if (!encode_fn()) return PA_ECUDA;
  pa_ctx* h = new pa_ctx();
  h->HQ = n_q_heads;
  h->HKV = n_kv_heads;
  h->G = G;
  h->TQ = kRows / G;
  h->n_pool = n_pool_pages;
  h->max_pages = max_pages_per_seq;
  h->opt = o;
  h->device = dev;
  h->n_sm = prop.multiProcessorCount;
  if (cudaMalloc(&h->d_err, kErrWords * sizeof(int)) != cudaSuccess ||
      cudaMemset(h->d_err, 0, kErrWords * sizeof(int)) != cudaSuccess ||
      cudaEventCreateWithFlags(&h->upload_done, cudaEventDisableTiming) != cudaSuccess) {
    pa_destroy(h);
    return PA_ECUDA;
  }
  *out = h;
  return PA_OK;
}

int pa_device(pa_handle h) { return h ? h->device : -1; }

void pa_destroy(pa_handle h) {
  if (!h) return;
  cudaDeviceSynchronize();
  void* ptrs[] = {h->kw, h->vt, h->ks, h->vs, h->vsmax, h->d_seqs, h->d_units, h->d_err, h->d_qflags, h->d_part,
                  h->d_tickets};
  for (void* p : ptrs)
    if (p) cudaFree(p);
  for (Workspace* w : {&h->sh_pre, &h->sh_own, &h->k4_part, &h->pages, &h->att_part}) {
    if (w->p) cudaFree(w->p);
    for (void* p : w->outgrown) cudaFree(p);
  }
  for (int i = 0; i < 7; ++i)
    if (h->hb[i]) cudaFree(h->hb[i]);
  if (h->h_stage) cudaFreeHost(h->h_stage);
  if (h->upload_done) cudaEventDestroy(h->upload_done);
  for (cudaEvent_t e : h->ev_free) cudaEventDestroy(e);
  for (cudaEvent_t e : h->ev_pending) cudaEventDestroy(e);
  for (cudaEvent_t e : h->pipe_ev) cudaEventDestroy(e);
  if (h->d_pseqs) cudaFree(h->d_pseqs);
  if (h->d_punits) cudaFree(h->d_punits);
  if (h->h_pstage) cudaFreeHost(h->h_pstage);
  if (h->pstage_done) cudaEventDestroy(h->pstage_done);
  if (h->s_h2d) cudaStreamDestroy(h->s_h2d);
  if (h->s_d2h) cudaStreamDestroy(h->s_d2h);
  delete h;
}

int pa_prefill(pa_handle h, const void* q, const int8_t* k_pool, const int8_t* v_pool, const float* k_scale,
               const float* v_scale, const int32_t* block_table, int q_start, int n_q, int n_ctx, int n_sink_blk,
               int n_win_blk, float sm_scale, void* out, void* stream) {
  pa_seq s{0, q_start, n_q, n_ctx};
  return run(h, 1, &s, q, k_pool, v_pool, k_scale, v_scale, block_table, n_sink_blk, n_win_blk, sm_scale, out,
             static_cast<cudaStream_t>(stream));
}

int pa_prefill_batch(pa_handle h, int n_seq, const pa_seq* seqs, const void* q, const int8_t* k_pool,
                     const int8_t* v_pool, const float* k_scale, const float* v_scale, const int32_t* block_table,
                     int n_sink_blk, int n_win_blk, float sm_scale, void* out, void* stream) {
  return run(h, n_seq, seqs, q, k_pool, v_pool, k_scale, v_scale, block_table, n_sink_blk, n_win_blk, sm_scale, out,
             static_cast<cudaStream_t>(stream));
}

int pa_prefill_batch_gated(pa_handle h, int n_seq, const pa_seq* seqs, const void* q, const void* q_gate,
                           const int8_t* k_pool, const int8_t* v_pool, const float* k_scale, const float* v_scale,
                           const int32_t* block_table, int n_sink_blk, int n_win_blk, float sm_scale, void* out,
                           void* stream) {
  if (!q_gate) return PA_EINVAL;
  return run(h, n_seq, seqs, q, k_pool, v_pool, k_scale, v_scale, block_table, n_sink_blk, n_win_blk, sm_scale, out,
             static_cast<cudaStream_t>(stream), q_gate);
}

// A piece of a sequence's query rows, computed as one call of its own.
// The host-buffer path is a pipeline over chunks of the query rows: the pool,
// scales and block table go in first and are widened once, then each chunk's
// q rows go in on one copy stream while the previous chunk is computed on the
// caller's stream and the one before that is copied out on another copy
// stream.  A chunk is a contiguous run of the sequences' rows laid end to
// end; a chunk boundary inside a sequence falls on a multiple of a work
// unit's tokens (256 / G, units start on those multiples), so every unit of
// the call's one plan belongs to exactly one chunk, and a chunk's attention
// launch runs just its units.
int pa_prefill_host(pa_handle h, int n_seq, const pa_seq* seqs, const void* q, const int8_t* k_pool,
                    const int8_t* v_pool, const float* k_scale, const float* v_scale, const int32_t* block_table,
                    int n_sink_blk, int n_win_blk, float sm_scale, void* out, void* stream) {
  if (!h || n_seq <= 0 || !seqs) return PA_EINVAL;
  // the whole call's plan validates it and sizes the widened workspace once
  Plan whole;
  int rc = build_plan(h->HQ, h->HKV, n_seq, seqs, n_sink_blk, n_win_blk, h->max_pages, whole);
  if (rc) return rc;
  const int total_q = whole.total_q;
  const size_t row_bytes = (size_t)h->HQ * kHeadDim * 2;  // one token's q (or out) row
  const size_t bytes[7] = {
      (size_t)total_q * row_bytes,                           // q
      (size_t)h->n_pool * kPage * h->HKV * kHeadDim,          // k_pool
      (size_t)h->n_pool * kPage * h->HKV * kHeadDim,          // v_pool
      (size_t)h->n_pool * kPage * h->HKV * sizeof(float),     // k_scale
      (size_t)h->n_pool * kPage * h->HKV * sizeof(float),     // v_scale
      (size_t)n_seq * h->max_pages * sizeof(int32_t),         // block table
      (size_t)total_q * row_bytes};                           // out
  const void* src[6] = {q, k_pool, v_pool, k_scale, v_scale, block_table};
  for (int i = 0; i < 6; ++i)
    if (!src[i]) return PA_EINVAL;
  if (!out) return PA_EINVAL;
  if (!(sm_scale == sm_scale) || sm_scale < 0.f) return PA_EINVAL;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  for (int i = 0; i < 7; ++i)
    if ((rc = grow_bytes(h->hb[i], h->hb_cap[i], bytes[i]))) return rc;

  // chunk boundaries on the sequences' rows laid end to end
  std::vector<long long> base(n_seq + 1, 0);  // first row of each sequence, end to end
  for (int s = 0; s < n_seq; ++s) base[s + 1] = base[s] + seqs[s].n_q;
  std::vector<long long> cuts;
  if ((rc = host_chunk_ends(h->HQ, h->HKV, n_seq, seqs, pa::attention_pairs(h->n_sm), cuts))) return rc;
  std::vector<std::vector<pa_seq>> chunks;  // per chunk, its pieces of the sequences (rows, same context)
  std::vector<long long> ends;  // chunk ends, end to end
  long long lo = 0;
  for (const long long hi : cuts) {
    if (hi <= lo) continue;
    chunks.emplace_back();
    ends.push_back(hi);
    for (int s = 0; s < n_seq; ++s) {
      const long long a = std::max(lo, base[s]), b = std::min(hi, base[s + 1]);
      if (a >= b) continue;
      const int qa = seqs[s].q_start + (int)(a - base[s]);
      chunks.back().push_back(pa_seq{seqs[s].q_off + (qa - seqs[s].q_start), qa, (int)(b - a), seqs[s].n_ctx});
    }
    lo = hi;
  }
  const int n_ch = (int)chunks.size();

  // one plan for the whole call (so one widening pass and the same per-sequence
  // V-scale maximum as pa_prefill_batch); its units split by chunk, each
  // chunk's list still in decreasing cost; all uploaded in one go ahead of the
  // large copies (a small copy queued behind them would hold up the first chunk)
  Plan P;
  if ((rc = build_plan(h->HQ, h->HKV, n_seq, seqs, n_sink_blk, n_win_blk, h->max_pages, P))) return rc;
  std::vector<std::vector<Unit>> cunits(n_ch);
  for (const Unit& u : P.units) {
    const pa_seq& q0 = seqs[u.seq];
    const long long row = base[u.seq] + (std::max(u.t0, q0.q_start) - q0.q_start);  // its first row, end to end
    const int c = (int)(std::upper_bound(ends.begin(), ends.end(), row) - ends.begin());
    if (c >= n_ch) return PA_EINVAL;  // cannot happen: every row lies in a chunk
    cunits[c].push_back(u);
  }
  // each chunk's units laid out pair by pair for its launch's pairs, the pair
  // offsets after them
  std::vector<std::vector<int>> coff(n_ch);
  std::vector<int> cpairs(n_ch, 0);
  std::vector<size_t> off_u(n_ch);
  size_t n_u = 0;
  for (int c = 0; c < n_ch; ++c) {
    const int n = (int)cunits[c].size();
    cpairs[c] = launch_pairs(h->n_sm, n);
    std::vector<Unit> by_pair;
    assign_pairs(cunits[c].data(), n, cpairs[c], by_pair, coff[c]);
    cunits[c] = std::move(by_pair);
    off_u[c] = n_u;
    n_u += (size_t)n + pair_off_records(cpairs[c]);
  }
  const size_t n_s = P.seqs.size();
  if ((rc = reserve_rows(h, (size_t)P.n_tok_total))) return rc;
  if ((rc = grow(h->vsmax, h->vsmax_cap, (size_t)n_seq * h->HKV))) return rc;
  if ((rc = grow(h->d_pseqs, h->pseqs_cap, n_s))) return rc;
  if ((rc = grow(h->d_punits, h->punits_cap, n_u))) return rc;
  if (!h->pstage_done) PA_CUDA(cudaEventCreateWithFlags(&h->pstage_done, cudaEventDisableTiming));
  if (h->pstage_recorded) PA_CUDA(cudaEventSynchronize(h->pstage_done));  // staging free again
  const size_t bytes_s = n_s * sizeof(SeqGeom), bytes_u = n_u * sizeof(Unit);
  if (h->h_pstage_cap < bytes_s + bytes_u) {
    if (h->h_pstage) cudaFreeHost(h->h_pstage);
    h->h_pstage = nullptr;
    h->h_pstage_cap = 0;
    PA_CUDA(cudaMallocHost(&h->h_pstage, bytes_s + bytes_u));
    h->h_pstage_cap = bytes_s + bytes_u;
  }
  std::memcpy(h->h_pstage, P.seqs.data(), bytes_s);
  for (int c = 0; c < n_ch; ++c) {
    Unit* dst = reinterpret_cast<Unit*>(static_cast<char*>(h->h_pstage) + bytes_s) + off_u[c];
    std::memcpy(dst, cunits[c].data(), cunits[c].size() * sizeof(Unit));
    std::memcpy(dst + cunits[c].size(), coff[c].data(), coff[c].size() * sizeof(int));
  }
  PA_CUDA(cudaMemcpyAsync(h->d_pseqs, h->h_pstage, bytes_s, cudaMemcpyHostToDevice, st));
  PA_CUDA(cudaMemcpyAsync(h->d_punits, static_cast<char*>(h->h_pstage) + bytes_s, bytes_u, cudaMemcpyHostToDevice, st));
  PA_CUDA(cudaEventRecord(h->pstage_done, st));
  h->pstage_recorded = true;

  // chunk c > 0 waits for its rows on the device (a flag the copy stream
  // writes after them), not with an event wait on the stream, so that its
  // launch can overlap the previous chunk's (programmatic dependent launch)
  const WriteValue32Fn write_value = write_value_fn();
  if (write_value && h->qflags_cap < n_ch) {
    if (h->d_qflags) cudaFree(h->d_qflags);
    h->d_qflags = nullptr;
    h->qflags_cap = 0;
    PA_CUDA(cudaMalloc(&h->d_qflags, (size_t)n_ch * sizeof(unsigned int)));
    PA_CUDA(cudaMemset(h->d_qflags, 0, (size_t)n_ch * sizeof(unsigned int)));
    h->qflags_cap = n_ch;
  }
  if (++h->q_epoch == 0) h->q_epoch = 1;  // flags start at 0: never a live epoch
  const unsigned int epoch = h->q_epoch;

  // streams and events
  if (!h->s_h2d) PA_CUDA(cudaStreamCreateWithFlags(&h->s_h2d, cudaStreamNonBlocking));
  if (!h->s_d2h) PA_CUDA(cudaStreamCreateWithFlags(&h->s_d2h, cudaStreamNonBlocking));
  const size_t n_ev = 3 + 2 * (size_t)n_ch;
  while (h->pipe_ev.size() < n_ev) {
    cudaEvent_t e;
    PA_CUDA(cudaEventCreateWithFlags(&e, cudaEventDisableTiming));
    h->pipe_ev.push_back(e);
  }
  cudaEvent_t ev_start = h->pipe_ev[0], ev_end = h->pipe_ev[1], ev_pool = h->pipe_ev[2];
  cudaEvent_t* ev_in = h->pipe_ev.data() + 3;           // chunk c's q rows are in
  cudaEvent_t* ev_done = h->pipe_ev.data() + 3 + n_ch;  // chunk c is computed

  // From the first copy on, the caller's host buffers are in use by copies on
  // the handle's streams: on any failure the call drains those streams (and
  // `stream`) before it returns, so no copy still reads q or the pool, or
  // writes out, once the caller gets control back.  Every chunk's row flag is
  // written before the first chunk launch, so the drain always ends.
  TimingMarks tm;
  auto enqueue = [&]() -> int {
    // inputs: after whatever the caller's stream did before
    PA_CUDA(cudaEventRecord(ev_start, st));
    PA_CUDA(cudaStreamWaitEvent(h->s_h2d, ev_start, 0));
    for (int i = 1; i < 6; ++i) PA_CUDA(cudaMemcpyAsync(h->hb[i], src[i], bytes[i], cudaMemcpyHostToDevice, h->s_h2d));
    PA_CUDA(cudaEventRecord(ev_pool, h->s_h2d));
    for (int c = 0; c < n_ch; ++c) {
      for (const pa_seq& pc : chunks[c]) {
        const size_t off = (size_t)pc.q_off * row_bytes;
        PA_CUDA(cudaMemcpyAsync(static_cast<char*>(h->hb[0]) + off, static_cast<const char*>(q) + off,
                                (size_t)pc.n_q * row_bytes, cudaMemcpyHostToDevice, h->s_h2d));
      }
      PA_CUDA(cudaEventRecord(ev_in[c], h->s_h2d));
      // test hook: a failure of the enqueue after the pool and the first rows are in flight
      if (h->opt.debug_fail_host && c == std::min(1, n_ch - 1)) return PA_ECUDA;
      if (write_value && c > 0 &&
          write_value(h->s_h2d, (CUdeviceptr)(h->d_qflags + c), epoch, CU_STREAM_WRITE_VALUE_DEFAULT) != CUDA_SUCCESS)
        return PA_ECUDA;
    }
    // widen the whole pool once it is in, then compute each chunk once its rows
    // are in; copy its output out behind it
    PA_CUDA(cudaStreamWaitEvent(h->s_d2h, ev_start, 0));
    PA_CUDA(cudaStreamWaitEvent(st, ev_pool, 0));
    int r = PA_OK;
    if (!(r = tm.init(h)) && !(r = tm.mark(h, 0, st)))
      r = launch_widen_plan(h, P, h->d_pseqs, n_seq, static_cast<const int8_t*>(h->hb[1]),
                            static_cast<const int8_t*>(h->hb[2]), static_cast<const float*>(h->hb[3]),
                            static_cast<const float*>(h->hb[4]), static_cast<const int32_t*>(h->hb[5]), sm_scale, st);
    if (!r) r = tm.mark(h, 1, st);
    if (r) return r;
    bool after_attn = false;  // the last launch on st is an attention launch of this call
    for (int c = 0; c < n_ch; ++c) {
      const bool on_device = write_value && c > 0 && after_attn;
      if (!on_device) PA_CUDA(cudaStreamWaitEvent(st, ev_in[c], 0));
      if (!cunits[c].empty()) {
        if ((r = launch_attention_plan(h, P, h->d_pseqs, h->d_punits + off_u[c], (int)cunits[c].size(), h->hb[0],
                                       n_sink_blk, n_win_blk, sm_scale, h->hb[6], st, nullptr, on_device,
                                       on_device ? h->d_qflags + c : nullptr, epoch,
                                       reinterpret_cast<const int*>(h->d_punits + off_u[c] + cunits[c].size()),
                                       cpairs[c])))
          return r;
        after_attn = true;
      }
      PA_CUDA(cudaEventRecord(ev_done[c], st));
      PA_CUDA(cudaStreamWaitEvent(h->s_d2h, ev_done[c], 0));
      for (const pa_seq& pc : chunks[c]) {
        const size_t off = (size_t)pc.q_off * row_bytes;
        PA_CUDA(cudaMemcpyAsync(static_cast<char*>(out) + off, static_cast<const char*>(h->hb[6]) + off,
                                (size_t)pc.n_q * row_bytes, cudaMemcpyDeviceToHost, h->s_d2h));
      }
    }
    if ((r = tm.mark(h, 2, st))) return r;
    // the caller's stream waits for both copy streams
    PA_CUDA(cudaEventRecord(ev_end, h->s_d2h));
    PA_CUDA(cudaStreamWaitEvent(st, ev_end, 0));
    PA_CUDA(cudaEventRecord(ev_start, h->s_h2d));
    PA_CUDA(cudaStreamWaitEvent(st, ev_start, 0));
    return PA_OK;
  };
  if ((rc = enqueue())) {
    tm.release(h);
    // errors of the drain itself are ignored: the first failure is reported
    (void)cudaStreamSynchronize(h->s_h2d);
    (void)cudaStreamSynchronize(h->s_d2h);
    (void)cudaStreamSynchronize(st);
    return rc;
  }
  return pa_last_error(h, stream);
}

int pa_debug_copy_streams_idle(pa_handle h) {
  if (!h) return PA_EINVAL;
  for (cudaStream_t s : {h->s_h2d, h->s_d2h}) {
    if (!s) continue;
    const cudaError_t e = cudaStreamQuery(s);
    if (e == cudaErrorNotReady) return 0;
    if (e != cudaSuccess) return PA_ECUDA;
  }
  return 1;
}

int pa_last_error(pa_handle h, void* stream) {
  if (!h) return PA_EINVAL;
  if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess) return PA_ECUDA;
  int e[kErrWords] = {};
  if (cudaMemcpy(e, h->d_err, sizeof e, cudaMemcpyDeviceToHost) != cudaSuccess) return PA_ECUDA;
  if ((e[0] | e[1]) != 0 && cudaMemset(h->d_err, 0, sizeof e) != cudaSuccess) return PA_ECUDA;
  if (e[0] & DEV_ERR_TIMEOUT) return PA_ETIMEOUT;
  if (e[0] != 0) return PA_ECUDA;
  if (e[1] != 0) return PA_EBADPAGE;
  return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ECUDA;
}

int pa_timing(pa_handle h, int reset, double* widen_ms, double* attention_ms, int* n_calls) {
  if (!h) return PA_EINVAL;
  for (size_t i = 0; i + 2 < h->ev_pending.size(); i += 3) {
    cudaEvent_t* e = &h->ev_pending[i];
    if (cudaEventSynchronize(e[2]) != cudaSuccess) return PA_ECUDA;
    float a = 0.f, b = 0.f;
    cudaEventElapsedTime(&a, e[0], e[1]);
    cudaEventElapsedTime(&b, e[1], e[2]);
    h->t_widen += a;
    h->t_attn += b;
    h->t_calls += 1;
    for (int k = 0; k < 3; ++k) h->ev_free.push_back(e[k]);
  }
  h->ev_pending.clear();
  if (widen_ms) *widen_ms = h->t_widen;
  if (attention_ms) *attention_ms = h->t_attn;
  if (n_calls) *n_calls = h->t_calls;
  if (reset) {
    h->t_widen = h->t_attn = 0.0;
    h->t_calls = 0;
  }
  return PA_OK;
}

int pa_plan(int n_q_heads, int n_kv_heads, int n_seq, const pa_seq* seqs, int n_sink_blk, int n_win_blk,
            int32_t* units_out, int cap, int* n_units, long long* n_tiles, int* n_widened_rows) {
  Plan P;
  int rc = build_plan(n_q_heads, n_kv_heads, n_seq, seqs, n_sink_blk, n_win_blk, 0, P);
  if (rc) return rc;
  if (n_units) *n_units = (int)P.units.size();
  if (n_tiles) *n_tiles = P.n_tiles;
  if (n_widened_rows) *n_widened_rows = P.n_tok_total;
  if (units_out) {
    const int n = std::min(cap, (int)P.units.size());
    for (int i = 0; i < n; ++i) {
      units_out[4 * i + 0] = P.units[i].seq;
      units_out[4 * i + 1] = P.units[i].g;
      units_out[4 * i + 2] = P.units[i].t0;
      units_out[4 * i + 3] = P.units[i].n_tiles;
    }
  }
  return PA_OK;
}

int pa_plan_pairs(int n_q_heads, int n_kv_heads, int n_seq, const pa_seq* seqs, int n_sink_blk, int n_win_blk,
                  int n_pairs, int32_t* units_out, int cap, int32_t* pair_off, int* n_units) {
  if (n_pairs < 1 || !pair_off) return PA_EINVAL;
  Plan P;
  int rc = build_plan(n_q_heads, n_kv_heads, n_seq, seqs, n_sink_blk, n_win_blk, 0, P);
  if (rc) return rc;
  const int n = (int)P.units.size();
  if (n_units) *n_units = n;
  if (units_out && cap < n) return PA_EINVAL;
  std::vector<Unit> by_pair;
  std::vector<int> off;
  assign_pairs(P.units.data(), n, n_pairs, by_pair, off);
  std::copy(off.begin(), off.end(), pair_off);
  if (units_out)
    for (int i = 0; i < n; ++i) {
      units_out[4 * i + 0] = by_pair[(size_t)i].seq;
      units_out[4 * i + 1] = by_pair[(size_t)i].g;
      units_out[4 * i + 2] = by_pair[(size_t)i].t0;
      units_out[4 * i + 3] = by_pair[(size_t)i].n_tiles;
    }
  return PA_OK;
}

int pa_host_chunks(int n_q_heads, int n_kv_heads, int n_seq, const pa_seq* seqs, int n_pairs, long long* chunk_end,
                   int cap, int* n_chunks) {
  std::vector<long long> ends;
  const int rc = host_chunk_ends(n_q_heads, n_kv_heads, n_seq, seqs, n_pairs, ends);
  if (rc) return rc;
  if (n_chunks) *n_chunks = (int)ends.size();
  if (chunk_end) {
    if ((int)ends.size() > cap) return PA_EINVAL;
    std::copy(ends.begin(), ends.end(), chunk_end);
  }
  return PA_OK;
}

int pa_debug_gather(pa_handle h, int n_seq, const pa_seq* seqs, const int8_t* k_pool, const int8_t* v_pool,
                    const float* k_scale, const float* v_scale, const int32_t* block_table, int n_sink_blk,
                    int n_win_blk, int seq, int8_t* k_out, int8_t* v_out, float* ks_out, float* vs_out,
                    int32_t* tok_out, int cap, int* n_rows, void* stream) {
  if (!h || !k_out || !v_out || !ks_out || !vs_out || !tok_out || !n_rows || seq < 0 || seq >= n_seq)
    return PA_EINVAL;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  int rc = prepare(h, n_seq, seqs, n_sink_blk, n_win_blk, st);
  if (rc) return rc;
  const int rows = h->plan.seqs[seq].n_blocks * kPage;
  *n_rows = rows;
  if (rows > cap) return PA_EINVAL;
  PA_CUDA(cudaMemsetAsync(h->vsmax, 0, sizeof(unsigned int) * n_seq * h->HKV, st));
  PA_CUDA(launch_widen(widen_params(h, k_pool, v_pool, k_scale, v_scale, block_table, n_seq), st));
  PA_CUDA(launch_debug_gather(widen_params(h, k_pool, v_pool, k_scale, v_scale, block_table, n_seq), seq, k_out,
                              v_out, ks_out, vs_out, tok_out, st));
  return pa_last_error(h, stream);
}

int pa_debug_qcodes(const void* q_rows, int n_rows, int8_t* codes, float* scales, void* stream) {
  if (n_rows < 0 || (n_rows > 0 && (!q_rows || !codes || !scales))) return PA_EINVAL;
  if (n_rows == 0) return PA_OK;
  if (!aligned(q_rows, 16) || !aligned(codes, 4) || !aligned(scales, 4)) return PA_EINVAL;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  PA_CUDA(launch_debug_qcodes(static_cast<const __nv_bfloat16*>(q_rows), n_rows, codes, scales, st));
  PA_CUDA(cudaStreamSynchronize(st));
  return PA_OK;
}

int pa_kv_append(pa_handle h, const void* k_new, const void* v_new, int n_new, int tok_start,
                 const int32_t* block_table_row, int8_t* k_pool, int8_t* v_pool, float* k_scale, float* v_scale,
                 void* stream) {
  if (!h || n_new < 0 || tok_start < 0) return PA_EINVAL;
  if (n_new == 0) return PA_OK;
  if (!k_new || !v_new || !block_table_row || !k_pool || !v_pool || !k_scale || !v_scale) return PA_EINVAL;
  if (!aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(k_pool, 16) || !aligned(v_pool, 16) ||
      !aligned(k_scale, 4) || !aligned(v_scale, 4) || !aligned(block_table_row, 4))
    return PA_EINVAL;
  if ((long long)tok_start + n_new > (long long)h->max_pages * kPage) return PA_EINVAL;
  KvAppendParams p{};
  p.k_new = static_cast<const __nv_bfloat16*>(k_new);
  p.v_new = static_cast<const __nv_bfloat16*>(v_new);
  p.n_new = n_new;
  p.tok_start = tok_start;
  p.HKV = h->HKV;
  p.n_pool = h->n_pool;
  p.bt_row = block_table_row;
  p.k_pool = k_pool;
  p.v_pool = v_pool;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.err = h->d_err;
  PA_CUDA(launch_kv_append(p, static_cast<cudaStream_t>(stream)));
  return PA_OK;
}

namespace {
// The handle's device is the current one inside the guard's scope.
struct OnDevice {
  int prev = -1;
  bool ok = true;
  explicit OnDevice(int device) {
    int cur = -1;
    if (cudaGetDevice(&cur) != cudaSuccess) ok = false;
    else if (cur != device) {
      ok = cudaSetDevice(device) == cudaSuccess;
      prev = cur;
    }
  }
  ~OnDevice() {
    if (prev >= 0) (void)cudaSetDevice(prev);
  }
};

// Bytes [lo, hi) of an array.
struct Span {
  uintptr_t lo = 0, hi = 0;
  bool meets(const Span& o) const { return lo < o.hi && o.lo < hi; }
};
Span span_of(const void* p, size_t bytes) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  return Span{a, a + bytes};
}

// Checks a host description of `tokens` rows of `heads` heads (row indexes
// below `tokens`) and fills the kernel's form and the bytes they lie in.
bool rows_ok(const pa_rows* r, long long tokens, int heads, RowsIn& in, Span& span) {
  if (!r || !r->data || !aligned(r->data, 16) || r->n_tok < tokens) return false;
  const long long ts = r->tok_stride, hs = r->head_stride;
  if (ts < 0 || hs < 0 || ts % 8 || hs % 8) return false;
  const long long most = 1ll << 46;  // elements: far above any device's memory, and no product below overflows
  if ((tokens > 1 && ts > most / tokens) || (heads > 1 && hs > most / heads)) return false;
  in = RowsIn{static_cast<const __nv_bfloat16*>(r->data), ts, hs};
  span = span_of(r->data, (size_t)((tokens - 1) * ts + (heads - 1) * hs + kHeadDim) * 2);
  return true;
}

// An output [tokens][heads][256] against the rows it is made from: apart, or the same rows in place.
bool out_ok(const Span& out, const Span& in, const RowsIn& rows, int heads, long long tokens) {
  if (!out.meets(in)) return true;
  return out.lo == in.lo && (heads == 1 || rows.hs == kHeadDim) &&
         (tokens == 1 || rows.ts == (long long)heads * kHeadDim);
}

bool rope_ok(const pa_rope* r) {
  if (r->rot_dim < 0 || r->rot_dim > kHeadDim || r->rot_dim % 16) return false;
  if (r->pairing != PA_ROPE_HALF && r->pairing != PA_ROPE_ADJACENT) return false;
  if (r->n_axes < 1 || r->n_axes > PA_ROPE_MAX_AXES) return false;
  for (int i = 0; i < r->rot_dim / 2; ++i)
    if (r->axis[i] >= r->n_axes) return false;
  return true;
}

// The arguments the two calls share: query and key rows of `tokens` row
// indexes, gains, eps, rotation, positions, the query's output.
struct QkvSpans {
  Span q, k, q_out;
  Span qw, kw, pos;  // empty where the kernel reads none
  bool read_beside_rows(const Span& out) const { return out.meets(qw) || out.meets(kw) || out.meets(pos); }
};
struct Heads {
  int HQ, HKV;
};
int qkv_common(const Heads& h, long long tokens, const pa_rows* q, const pa_rows* k, const void* qw, const void* kw,
               float w_off, float eps, const pa_rope* rope, const int32_t* pos, long long pos_stride, void* q_out,
               QkvParams& p, QkvSpans& sp) {
  if ((q == nullptr) != (q_out == nullptr)) return PA_EINVAL;
  if (!std::isfinite(eps) || eps < 0.f || !std::isfinite(w_off)) return PA_EINVAL;
  if (qw && !aligned(qw, 16)) return PA_EINVAL;
  if (kw && !aligned(kw, 16)) return PA_EINVAL;
  if (q) {
    if (!rows_ok(q, tokens, h.HQ, p.q, sp.q) || !aligned(q_out, 16)) return PA_EINVAL;
    sp.q_out = span_of(q_out, (size_t)tokens * h.HQ * kHeadDim * 2);
    if (!out_ok(sp.q_out, sp.q, p.q, h.HQ, tokens)) return PA_EINVAL;
    p.n_q = h.HQ;
  }
  if (k) {
    if (!rows_ok(k, tokens, h.HKV, p.k, sp.k)) return PA_EINVAL;
    if (q && sp.q_out.meets(sp.k)) return PA_EINVAL;
    p.n_k = h.HKV;
  }
  p.qw = static_cast<const __nv_bfloat16*>(qw);
  p.kw = static_cast<const __nv_bfloat16*>(kw);
  p.w_off = w_off;
  p.eps = eps;
  p.rope.n_axes = 1;
  if (rope) {
    if (!rope_ok(rope)) return PA_EINVAL;
    p.rope = *rope;
  }
  if (p.rope.rot_dim > 0 && pos) {
    if (!aligned(pos, 4) || pos_stride < 0 || (p.rope.n_axes > 1 && (pos_stride < tokens || pos_stride > 1ll << 46)))
      return PA_EINVAL;
    p.pos = pos;
    p.pos_stride = pos_stride;
    sp.pos = span_of(pos, (size_t)((p.rope.n_axes - 1) * pos_stride + tokens) * sizeof(int32_t));
  }
  if (q && qw) sp.qw = span_of(qw, kHeadDim * 2);
  if (k && kw) sp.kw = span_of(kw, kHeadDim * 2);
  if (q && sp.read_beside_rows(sp.q_out)) return PA_EINVAL;
  p.q_out = static_cast<__nv_bfloat16*>(q_out);
  return PA_OK;
}

// Whether two sequences of a batch have a row in common.
bool rows_shared(int n_seq, const pa_seq* seqs) {
  bool sorted = true;
  for (int s = 1; s < n_seq && sorted; ++s) sorted = seqs[s].q_off >= seqs[s - 1].q_off + seqs[s - 1].n_q;
  if (sorted) return false;
  std::vector<std::pair<int, int>> r((size_t)n_seq);
  for (int s = 0; s < n_seq; ++s) r[(size_t)s] = {seqs[s].q_off, seqs[s].q_off + seqs[s].n_q};
  std::sort(r.begin(), r.end());
  for (size_t s = 1; s < r.size(); ++s)
    if (r[s].first < r[s - 1].second) return true;
  return false;
}

// Arguments of pa_qk_norm_rope (n_tok >= 1) -> the kernel's parameters.
int qk_norm_rope_args(const Heads& h, int n_tok, const pa_rows* q, const pa_rows* k, const void* qw, const void* kw,
                      float w_off, float eps, const pa_rope* rope, const int32_t* pos, long long pos_stride,
                      void* q_out, void* k_out, QkvParams& p) {
  if ((!q && !k) || (k == nullptr) != (k_out == nullptr)) return PA_EINVAL;
  QkvSpans sp;
  const int rc = qkv_common(h, n_tok, q, k, qw, kw, w_off, eps, rope, pos, pos_stride, q_out, p, sp);
  if (rc) return rc;
  if (p.rope.rot_dim > 0 && !p.pos) return PA_EINVAL;
  if (k) {
    if (!aligned(k_out, 16)) return PA_EINVAL;
    const Span ko = span_of(k_out, (size_t)n_tok * h.HKV * kHeadDim * 2);
    if (!out_ok(ko, sp.k, p.k, h.HKV, n_tok)) return PA_EINVAL;
    if ((q && (ko.meets(sp.q) || ko.meets(sp.q_out))) || sp.read_beside_rows(ko)) return PA_EINVAL;
    p.k_out = static_cast<__nv_bfloat16*>(k_out);
  }
  p.n_tok = n_tok;
  return PA_OK;
}

// Arguments of pa_qkv_append (n_seq >= 1) -> the kernel's parameters, but for each launch's sequences.
// n_pool 0: the pools' sizes are not known, and overlaps with them not looked for.
int qkv_append_args(const Heads& h, int n_pool, int max_pages, int n_seq, const pa_seq* seqs, const pa_rows* q, const pa_rows* k,
                    const pa_rows* v, const void* qw, const void* kw, float w_off, float eps, const pa_rope* rope,
                    const int32_t* pos, long long pos_stride, const int32_t* bt, int8_t* kp, int8_t* vp, float* ksc,
                    float* vsc, void* q_out, QkvParams& p) {
  if (!seqs || !k || !v || !bt || !kp || !vp || !ksc || !vsc) return PA_EINVAL;
  if (!aligned(kp, 16) || !aligned(vp, 16) || !aligned(ksc, 4) || !aligned(vsc, 4) || !aligned(bt, 4))
    return PA_EINVAL;
  long long tokens = 0;  // rows of the arrays
  for (int s = 0; s < n_seq; ++s) {
    const pa_seq& a = seqs[s];
    if (a.n_q < 1 || a.q_start < 0 || a.q_off < 0 || (long long)a.q_start + a.n_q > a.n_ctx ||
        (long long)a.q_start + a.n_q > (long long)max_pages * kPage || (long long)a.q_off + a.n_q > (1ll << 30))
      return PA_EINVAL;
    tokens = std::max(tokens, (long long)a.q_off + a.n_q);
  }
  if (rows_shared(n_seq, seqs)) return PA_EINVAL;
  QkvSpans sp;
  const int rc = qkv_common(h, tokens, q, k, qw, kw, w_off, eps, rope, pos, pos_stride, q_out, p, sp);
  if (rc) return rc;
  Span vs;
  if (!rows_ok(v, tokens, h.HKV, p.v, vs) || (q && sp.q_out.meets(vs))) return PA_EINVAL;
  const Span table = span_of(bt, (size_t)n_seq * max_pages * sizeof(int32_t));
  if (q && sp.q_out.meets(table)) return PA_EINVAL;
  if (n_pool > 0) {
    const size_t slots = (size_t)n_pool * kPage * h.HKV;
    const Span pool[4] = {span_of(kp, slots * kHeadDim), span_of(vp, slots * kHeadDim), span_of(ksc, slots * sizeof(float)),
                          span_of(vsc, slots * sizeof(float))};
    for (int i = 0; i < 4; ++i) {
      const Span& w = pool[i];
      if (w.meets(sp.q) || w.meets(sp.k) || w.meets(vs) || w.meets(table) || sp.read_beside_rows(w)) return PA_EINVAL;
      if (w.meets(sp.q_out)) return PA_EINVAL;
      for (int j = 0; j < i; ++j)
        if (w.meets(pool[j])) return PA_EINVAL;
    }
  }
  p.n_v = h.HKV;
  p.block_table = bt;
  p.bt_stride = max_pages;
  p.HKV = h.HKV;
  p.k_pool = kp;
  p.v_pool = vp;
  p.k_scale = ksc;
  p.v_scale = vsc;
  return PA_OK;
}

// A launch over n_tok tokens: how many rows a warp takes.
void qkv_split(QkvParams& p, int n_tok, int n_sm) {
  const int rows = p.n_q + p.n_k + p.n_v;
  p.n_tok = n_tok;
  p.rows_per_part = qkv_rows_per_part(n_tok, rows, n_sm);
  p.parts = (rows + p.rows_per_part - 1) / p.rows_per_part;
}

bool heads_ok(int HQ, int HKV) {  // pa_create's requirements
  return HQ > 0 && HKV > 0 && HKV <= 8 && HQ % HKV == 0 && HQ / HKV <= kRows && kRows % (HQ / HKV) == 0;
}
}  // namespace

namespace {
// inv_freq / (2 pi) modulo 1, times 2^64, to the nearest integer (|inv_freq| < 2^64):
// the double's 53 bits times 1 / (2 pi) to 256 bits, from which 2^64 takes 117 at most.
uint64_t turn_of(double inv_freq) {
  static constexpr uint64_t kInv2Pi[4] = {0x28be60db9391054aull, 0x7f09d5f47d4d3770ull, 0x36d8a5664f10e410ull,
                                          0x7f9458eaf7aef158ull};  // 2^-64, 2^-128, ...
  int e = 0;
  const uint64_t m = (uint64_t)std::ldexp(std::frexp(std::fabs(inv_freq), &e), 53);
  e -= 53;  // |inv_freq| = m 2^e
  uint64_t p[6] = {};  // m times the 256-bit integer, lowest word first
  unsigned __int128 carry = 0;
  for (int i = 0; i < 4; ++i) {
    carry += (unsigned __int128)m * kInv2Pi[3 - i];
    p[i] = (uint64_t)carry;
    carry >>= 64;
  }
  p[4] = (uint64_t)carry;
  // the turns are p 2^(e - 256): their fraction's first 64 bits, and the next one to round by
  const int s = 192 - e;  // at least 181
  auto bits64 = [&](int at) -> uint64_t {
    const int w = at >> 6, b = at & 63;
    if (w > 4) return 0;
    return p[w] >> b | (b ? p[w + 1] << (64 - b) : 0);
  };
  const uint64_t turn = bits64(s) + (bits64(s - 1) & 1);
  return inv_freq < 0.0 ? 0 - turn : turn;
}
}  // namespace

int pa_rope_init(pa_rope* rope, int rot_dim, int pairing, int n_axes, const double* inv_freq,
                 const int32_t* pair_axis) {
  if (!rope || rot_dim < 0 || rot_dim > kHeadDim || rot_dim % 16 || n_axes < 1 || n_axes > PA_ROPE_MAX_AXES ||
      (pairing != PA_ROPE_HALF && pairing != PA_ROPE_ADJACENT) || (rot_dim > 0 && !inv_freq))
    return PA_EINVAL;
  pa_rope r;
  std::memset(&r, 0, sizeof r);
  r.rot_dim = rot_dim;
  r.pairing = pairing;
  r.n_axes = n_axes;
  for (int i = 0; i < rot_dim / 2; ++i) {
    const int a = pair_axis ? pair_axis[i] : 0;
    if (a < 0 || a >= n_axes || !(std::fabs(inv_freq[i]) < 18446744073709551616.0)) return PA_EINVAL;  // 2^64; NaN
    r.axis[i] = (uint8_t)a;
    r.turn[i] = turn_of(inv_freq[i]);
  }
  *rope = r;
  return PA_OK;
}

int pa_qk_norm_rope(pa_handle h, int n_tok, const pa_rows* q, const pa_rows* k, const void* q_weight,
                    const void* k_weight, float weight_offset, float eps, const pa_rope* rope,
                    const int32_t* positions, long long pos_stride, void* q_out, void* k_out, void* stream) {
  if (!h || n_tok < 0 || n_tok > (1 << 30)) return PA_EINVAL;
  if (n_tok == 0) return PA_OK;
  QkvParams p{};
  const int rc = qk_norm_rope_args(Heads{h->HQ, h->HKV}, n_tok, q, k, q_weight, k_weight, weight_offset, eps, rope,
                                   positions, pos_stride, q_out, k_out, p);
  if (rc) return rc;
  qkv_split(p, n_tok, h->n_sm);
  OnDevice dev(h->device);
  if (!dev.ok) return PA_ECUDA;
  PA_CUDA(launch_qk_norm_rope(p, h->n_sm, static_cast<cudaStream_t>(stream)));
  return PA_OK;
}

int pa_qkv_append(pa_handle h, int n_seq, const pa_seq* seqs, const pa_rows* q, const pa_rows* k, const pa_rows* v,
                  const void* q_weight, const void* k_weight, float weight_offset, float eps, const pa_rope* rope,
                  const int32_t* positions, long long pos_stride, const int32_t* block_table, int8_t* k_pool,
                  int8_t* v_pool, float* k_scale, float* v_scale, void* q_out, void* stream) {
  if (!h || n_seq < 0) return PA_EINVAL;
  if (n_seq == 0) return PA_OK;
  QkvParams p{};
  const int rc = qkv_append_args(Heads{h->HQ, h->HKV}, h->n_pool, h->max_pages, n_seq, seqs, q, k, v, q_weight, k_weight,
                                 weight_offset, eps, rope, positions, pos_stride, block_table, k_pool, v_pool,
                                 k_scale, v_scale, q_out, p);
  if (rc) return rc;
  p.n_pool = h->n_pool;
  p.err = h->d_err;
  OnDevice dev(h->device);
  if (!dev.ok) return PA_ECUDA;
  QkvSeqs<kQkvSeqs> tab;
  for (int s0 = 0; s0 < n_seq; s0 += kQkvSeqs) {
    const int n = std::min(kQkvSeqs, n_seq - s0);
    int first = 0;
    p.same_len = seqs[s0].n_q;
    for (int i = 0; i < n; ++i) {
      const pa_seq& a = seqs[s0 + i];
      tab.s[i] = make_int4(a.q_off, a.q_start, first, 0);
      first += a.n_q;  // at most 2^30: the sequences' rows are disjoint
      if (a.n_q != p.same_len) p.same_len = 0;
    }
    p.n_seq = n;
    p.bt_row0 = s0;
    qkv_split(p, first, h->n_sm);
    PA_CUDA(launch_qkv_append(p, tab, h->n_sm, static_cast<cudaStream_t>(stream)));
  }
  return PA_OK;
}

int pa_debug_qk_norm_rope_check(int n_q_heads, int n_kv_heads, int n_tok, const pa_rows* q, const pa_rows* k,
                                const void* q_weight, const void* k_weight, float weight_offset, float eps,
                                const pa_rope* rope, const int32_t* positions, long long pos_stride, void* q_out,
                                void* k_out) {
  if (!heads_ok(n_q_heads, n_kv_heads) || n_tok < 0 || n_tok > (1 << 30)) return PA_EINVAL;
  if (n_tok == 0) return PA_OK;
  QkvParams p{};
  return qk_norm_rope_args(Heads{n_q_heads, n_kv_heads}, n_tok, q, k, q_weight, k_weight, weight_offset, eps, rope,
                           positions, pos_stride, q_out, k_out, p);
}

int pa_debug_qkv_append_pool_check(int n_q_heads, int n_kv_heads, int n_pool_pages, int max_pages_per_seq, int n_seq,
                                   const pa_seq* seqs, const pa_rows* q, const pa_rows* k, const pa_rows* v,
                                   const void* q_weight, const void* k_weight, float weight_offset, float eps,
                                   const pa_rope* rope, const int32_t* positions, long long pos_stride,
                                   const int32_t* block_table, int8_t* k_pool, int8_t* v_pool, float* k_scale,
                                   float* v_scale, void* q_out) {
  if (!heads_ok(n_q_heads, n_kv_heads) || n_seq < 0 || n_pool_pages < 0) return PA_EINVAL;
  if (n_seq == 0) return PA_OK;
  QkvParams p{};
  return qkv_append_args(Heads{n_q_heads, n_kv_heads}, n_pool_pages, max_pages_per_seq, n_seq, seqs, q, k, v, q_weight,
                         k_weight, weight_offset, eps, rope, positions, pos_stride, block_table, k_pool, v_pool, k_scale,
                         v_scale, q_out, p);
}

int pa_debug_qkv_append_check(int n_q_heads, int n_kv_heads, int max_pages_per_seq, int n_seq, const pa_seq* seqs,
                              const pa_rows* q, const pa_rows* k, const pa_rows* v, const void* q_weight,
                              const void* k_weight, float weight_offset, float eps, const pa_rope* rope,
                              const int32_t* positions, long long pos_stride, const int32_t* block_table,
                              int8_t* k_pool, int8_t* v_pool, float* k_scale, float* v_scale, void* q_out) {
  return pa_debug_qkv_append_pool_check(n_q_heads, n_kv_heads, 0, max_pages_per_seq, n_seq, seqs, q, k, v, q_weight,
                                        k_weight, weight_offset, eps, rope, positions, pos_stride, block_table, k_pool,
                                        v_pool, k_scale, v_scale, q_out);
}

namespace {
// Cost-balanced decode runs over a launch's pair list (block counts `len`,
// HKV pairs per sequence).  A CTA costs its blocks plus kDecSegCost for every
// pair after its first: a run that crosses into another pair waits for all
// its warps, combines them, loads the next pair's query rows and refills its
// copies (measured at 64 sequences x 32k context: such CTAs ended ~10 us,
// about 16 blocks' worth, after the others).  Greedy packing under `budget`;
// false if it needs more than max_ctas CTAs.
constexpr int kDecSegCost = 16;
bool decode_pack(const std::vector<int>& len, int HKV, long long total, long long budget, long long max_ctas,
                 DecRuns& r) {
  r.x0.clear();
  r.seq.clear();
  r.slot.clear();
  r.max_slots = 1;
  std::vector<int> first_cta(len.size(), 0);
  size_t pi = 0;
  long long pstart = 0, x = 0;
  int cta = 0;
  while (x < total) {
    if (cta >= max_ctas) return false;
    r.x0.push_back((int)x);
    r.seq.push_back((int)(pi / (size_t)HKV));
    r.slot.push_back(x == pstart ? 0 : cta - first_cta[pi]);
    long long cost = 0;
    bool first = true;
    while (x < total) {
      const long long pend = pstart + len[pi];
      const long long extra = first ? 0 : kDecSegCost;
      if (cost + extra >= budget) break;
      if (x == pstart) first_cta[pi] = cta;
      const long long take = std::min(pend - x, budget - cost - extra);
      cost += extra + take;
      x += take;
      first = false;
      if (x < pend) break;  // the budget ran out inside the pair
      r.max_slots = std::max(r.max_slots, cta - first_cta[pi] + 1);
      ++pi;
      pstart = pend;
    }
    ++cta;
  }
  return true;
}

// Visible blocks of a decode query (the context's last token, t = n_ctx - 1)
// under the prefill's block mask: sink blocks, then the window run up to t's block.
int decode_n_vis(int n_ctx, int n_sink_blk, int n_win_blk) {
  const int last = (n_ctx - 1) / kPage;
  const int lo = n_win_blk > 0 ? std::max(0, last + 1 - n_win_blk) : 0;
  const int n_sink = n_win_blk > 0 ? std::min(std::max(n_sink_blk, 0), lo) : 0;
  return n_sink + (last - lo + 1);
}

// One decode launch (up to kDecParamSeqs sequences): the launch's pairs'
// blocks end to end; one wave of cost-balanced runs listed in the parameters
// when runs of at most 128 blocks fit in one wave, else whole waves of equal
// runs of per_cta blocks.
struct DecLaunch {
  int s0 = 0, n = 0, total = 0, per_cta = 0, n_cta = 0, max_slots = 1;
  bool listed = false;
  DecRuns runs;
};
int decode_launch_plan(int HKV, long long slots, const int* n_vis, int s0, int n, DecLaunch& L) {
  L = DecLaunch{};
  L.s0 = s0;
  L.n = n;
  long long vis = 0;
  int nv_max = 1;
  std::vector<int> len;
  for (int i = 0; i < n; ++i) {
    vis += n_vis[i];
    nv_max = std::max(nv_max, n_vis[i]);
    for (int g = 0; g < HKV; ++g) len.push_back(n_vis[i]);
  }
  const long long total = vis * HKV;
  if (total >= (1ll << 30) || slots < 1) return PA_EINVAL;
  L.total = (int)total;
  const long long wave = std::min<long long>(slots, kDecParamCtas);
  if (total <= wave * kDecMaxCtaBlocks && decode_pack(len, HKV, total, kDecMaxCtaBlocks, wave, L.runs)) {
    long long lo = std::max(1ll, (total + wave - 1) / wave), hi = kDecMaxCtaBlocks;
    while (lo < hi) {  // the smallest budget that packs into one wave
      const long long mid = (lo + hi) / 2;
      if (decode_pack(len, HKV, total, mid, wave, L.runs)) hi = mid;
      else lo = mid + 1;
    }
    (void)decode_pack(len, HKV, total, lo, wave, L.runs);
    L.listed = true;
    L.per_cta = (int)lo;
    L.n_cta = (int)L.runs.x0.size();
    L.max_slots = L.runs.max_slots;
  } else {
    const long long full = (total + kDecMaxCtaBlocks - 1) / kDecMaxCtaBlocks;
    const long long waves = std::max(1ll, (full + slots - 1) / slots);
    L.listed = false;
    L.per_cta = (int)std::max(1ll, (total + waves * slots - 1) / (waves * slots));
    L.n_cta = (int)((total + L.per_cta - 1) / L.per_cta);
    L.max_slots = (nv_max - 1 + L.per_cta - 1) / L.per_cta + 1;  // CTA runs a pair's blocks can meet
  }
  return PA_OK;
}

// A decode query's checks: one token, the context's last, within the block table.
bool decode_seq_ok(const pa_seq& q1, int max_pages) {
  return q1.n_q == 1 && q1.q_off >= 0 && q1.n_ctx >= 1 && q1.q_start == q1.n_ctx - 1 &&
         (q1.n_ctx + kPage - 1) / kPage <= max_pages;
}
}  // namespace

int pa_decode_plan(int n_kv_heads, int slots, int n_seq, const pa_seq* seqs, int n_sink_blk, int n_win_blk,
                   int32_t* runs_out, int cap, int* n_cta, int* per_cta, int* max_slots, int* listed,
                   long long* total_blocks) {
  if (n_kv_heads < 1 || n_kv_heads > 8 || slots < 1 || n_seq <= 0 || !seqs) return PA_EINVAL;
  const int n = std::min(n_seq, kDecParamSeqs);
  std::vector<int> n_vis((size_t)n);
  for (int s = 0; s < n; ++s) {
    if (!decode_seq_ok(seqs[s], INT32_MAX)) return PA_EINVAL;
    n_vis[(size_t)s] = decode_n_vis(seqs[s].n_ctx, n_sink_blk, n_win_blk);
  }
  DecLaunch L;
  const int rc = decode_launch_plan(n_kv_heads, slots, n_vis.data(), 0, n, L);
  if (rc) return rc;
  if (n_cta) *n_cta = L.n_cta;
  if (per_cta) *per_cta = L.per_cta;
  if (max_slots) *max_slots = L.max_slots;
  if (listed) *listed = L.listed ? 1 : 0;
  if (total_blocks) *total_blocks = L.total;
  if (runs_out) {
    if (cap < L.n_cta) return PA_EINVAL;
    if (L.listed) {
      for (int c = 0; c < L.n_cta; ++c) {
        runs_out[3 * c] = L.runs.x0[(size_t)c];
        runs_out[3 * c + 1] = L.runs.seq[(size_t)c];
        runs_out[3 * c + 2] = L.runs.slot[(size_t)c];
      }
    } else {  // equal runs: CTA c starts at c per_cta; its slot counts the CTAs before it in that block's pair
      long long pstart = 0;
      int s = 0, g = 0;
      for (int c = 0; c < L.n_cta; ++c) {
        const long long x = (long long)c * L.per_cta;
        while (x >= pstart + n_vis[(size_t)s]) {
          pstart += n_vis[(size_t)s];
          if (++g == n_kv_heads) {
            g = 0;
            ++s;
          }
        }
        runs_out[3 * c] = (int)x;
        runs_out[3 * c + 1] = s;
        runs_out[3 * c + 2] = c - (int)(pstart / L.per_cta);
      }
    }
  }
  return PA_OK;
}

namespace {
// The pool as uint8 [n_pool * 16][HKV][256]; a box is one kv head's 16 token rows of half the dims.
int pool_maps(pa_handle h, const int8_t* k_pool, const int8_t* v_pool, DecodeMaps& m) {
  const uint64_t dims[3] = {(uint64_t)kHeadDim, (uint64_t)h->HKV, (uint64_t)h->n_pool * kPage};
  const uint64_t strides[2] = {(uint64_t)kHeadDim, (uint64_t)h->HKV * kHeadDim};
  const uint32_t box[3] = {128, 1, (uint32_t)kPage};
  const int rc = encode(&m.k, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, k_pool, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
  return rc ? rc : encode(&m.v, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, v_pool, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}
}  // namespace

int pa_decode(pa_handle h, int n_seq, const pa_seq* seqs, const void* q, const int8_t* k_pool, const int8_t* v_pool,
              const float* k_scale, const float* v_scale, const int32_t* block_table, int n_sink_blk, int n_win_blk,
              float sm_scale, void* out, void* stream) {
  int rc = check_inputs(h, q, k_pool, v_pool, k_scale, v_scale, block_table, out);
  if (rc) return rc;
  if (n_seq <= 0 || !seqs || h->G > 8 || !(sm_scale == sm_scale) || sm_scale < 0.f) return PA_EINVAL;
  std::vector<int> n_vis((size_t)n_seq);
  for (int s = 0; s < n_seq; ++s) {
    if (!decode_seq_ok(seqs[s], h->max_pages)) return PA_EINVAL;
    n_vis[(size_t)s] = decode_n_vis(seqs[s].n_ctx, n_sink_blk, n_win_blk);
  }
  // launches of up to kDecParamSeqs sequences, their table in the launch's parameters
  std::vector<DecLaunch> launches;
  const long long slots = (long long)h->n_sm * decode_ctas_per_sm(h->HKV);
  size_t part_need = 0;
  for (int s0 = 0; s0 < n_seq; s0 += kDecParamSeqs) {
    DecLaunch L;
    if ((rc = decode_launch_plan(h->HKV, slots, n_vis.data() + s0, s0, std::min(kDecParamSeqs, n_seq - s0), L)))
      return rc;
    part_need = std::max(part_need, (size_t)L.n * h->HKV * L.max_slots * h->G * kDecPartStride);
    launches.push_back(std::move(L));
  }
  if (part_need > (size_t)INT32_MAX) return PA_EINVAL;
  if ((rc = grow(h->d_part, h->part_cap, part_need))) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (h->tickets_cap < kDecParamSeqs * h->HKV) {
    if ((rc = grow(h->d_tickets, h->tickets_cap, (size_t)kDecParamSeqs * h->HKV))) return rc;
    PA_CUDA(cudaMemsetAsync(h->d_tickets, 0, (size_t)h->tickets_cap * sizeof(unsigned long long), st));
  }
  if (k_pool != h->dec_kp || v_pool != h->dec_vp) {
    h->dec_kp = h->dec_vp = nullptr;
    if ((rc = pool_maps(h, k_pool, v_pool, h->dec_maps))) return rc;
    h->dec_kp = k_pool;
    h->dec_vp = v_pool;
  }
  DecodeParams p{};
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.out = static_cast<__nv_bfloat16*>(out);
  p.k_pool = k_pool;
  p.v_pool = v_pool;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.block_table = block_table;
  p.bt_stride = h->max_pages;
  p.n_pool = h->n_pool;
  p.S = n_sink_blk;
  p.W = n_win_blk;
  p.HQ = h->HQ;
  p.HKV = h->HKV;
  p.G = h->G;
  p.sm_scale_log2 = sm_scale * 1.4426950408889634f;
  p.part = h->d_part;
  p.tickets = h->d_tickets;
  p.err = h->d_err;
  p.wait_ns = (unsigned long long)h->opt.wait_timeout_ms * 1000000ull;
  DecodeSeqs tab;
  for (const DecLaunch& L : launches) {
    int vstart = 0;
    for (int i = 0; i < L.n; ++i) {
      const pa_seq& q1 = seqs[L.s0 + i];
      tab.seq[i] = make_int4(q1.q_off, q1.n_ctx, vstart, 0);
      vstart += n_vis[(size_t)(L.s0 + i)];
    }
    p.n_seq = L.n;
    p.bt_row0 = L.s0;
    p.total = L.total;
    p.per_cta = L.per_cta;
    p.max_slots = L.max_slots;
    p.runs_listed = L.listed ? 1 : 0;
    if (L.listed)
      for (int c = 0; c < L.n_cta; ++c) {
        tab.cta_x0[c] = L.runs.x0[(size_t)c];
        tab.cta_seq[c] = (uint16_t)L.runs.seq[(size_t)c];
        tab.cta_slot[c] = (uint16_t)L.runs.slot[(size_t)c];
      }
    PA_CUDA(launch_decode(p, tab, h->dec_maps, L.n_cta, st));
  }
  return PA_OK;
}

namespace {
int decode_shared_check(int HQ, int HKV, int max_pages, int n_seq, const pa_seq* seqs, int n_prefix, int S,
                        float sm_scale) {
  if (!heads_ok(HQ, HKV) || HQ / HKV > 8 || n_seq < 1 || !seqs || S < 0) return PA_EINVAL;
  if (!std::isfinite(sm_scale) || sm_scale < 0.f) return PA_EINVAL;
  if (n_prefix < 0 || n_prefix % kPage || (n_prefix > 0 && n_prefix / kPage > max_pages)) return PA_EINVAL;
  for (int s = 0; s < n_seq; ++s)
    if (!decode_seq_ok(seqs[s], max_pages) || seqs[s].n_ctx <= n_prefix || seqs[s].n_ctx > (1 << 30) ||
        seqs[s].q_off >= (1 << 30))
      return PA_EINVAL;
  return rows_shared(n_seq, seqs) ? PA_EINVAL : PA_OK;
}

// One launch (sequences [s0, s0 + n)) of the shared-prefix decode: its table and split.
// The prefix pass: up to 128 rows of a kv head (n sequences x G) are one CTA's; more
// are worked on by pairs of CTAs, in groups of 256.  Per group the blocks some row
// sees, in 128-key tiles; all tiles, group after group, cut
// into runs of equal cost, one for each unit (a CTA or a pair, one CTA an SM).  A
// run costs its tiles plus kShSegCost for every group after its first: the next
// group's queries are staged and the last one's output stored while no product
// runs (about 12000 cycles against 3000 to 4000 a pair's tile on GB300).  The
// per-sequence pass: chunks of equal block counts, four to 128 blocks each.
constexpr int kShSegCost = 4, kShOwnWaves = 2;
// Microseconds on GB300, fitted to 27 batches at 5 to 14 numbers of units each: a
// unit's set-up, queries and epilogue, its first ten tiles, the others, and what
// the per-sequence pass adds when it ends after the prefix pass; a tile's factor
// where windows mask keys; the SM time of an own block, of a prefix block that a
// sequence reads again (from L2) and of an own CTA, what the per-sequence pass
// takes to get going, and how full it keeps its SMs when not even a CTA for every
// sequence fits them at once.
struct ShCost {
  double unit, tile, late, tail;
};
constexpr ShCost kShCost[2] = {{11.5, 2.5, 2.65, 2.0}, {11.0, 2.1, 1.65, 4.0}};  // units of one CTA, of two
constexpr double kShMaskedTile = 1.25;
constexpr double kShOwnBlockUs = 0.215, kShAgainBlockUs = 0.165, kShOwnCtaUs = 0.25;
constexpr double kShOwnStartUs = 4.5, kShOwnFull = 0.85;
// Packs the groups (nt[j] tiles each, laid end to end) into runs of at most
// `budget` cost; false if they take more than max_units.
bool shared_pack(const int* nt, int n_groups, int budget, int max_units, int* cut, int& n_units) {
  int c = 0, cost = 0, x = 0;
  cut[0] = 0;
  for (int j = 0; j < n_groups; ++j) {
    int left = nt[j];
    while (left > 0) {
      const int extra = cost > 0 ? kShSegCost : 0;
      if (cost + extra >= budget) {  // the run is full
        if (++c >= max_units) return false;
        cut[c] = x;
        cost = 0;
        continue;
      }
      const int take = std::min(left, budget - cost - extra);
      cost += extra + take;
      x += take;
      left -= take;
    }
  }
  n_units = c + 1;
  cut[n_units] = x;
  return true;
}

int decode_shared_plan(int HQ, int HKV, int n_sm, const pa_seq* seqs, int s0, int n, int n_prefix, int S, int W,
                       int prefix_pass, SharedParams& p, SharedSeqs& t) {
  const int G = HQ / HKV, Pb = n_prefix / kPage;
  p.n_seq = n;
  p.bt_row0 = s0;
  p.HQ = HQ;
  p.HKV = HKV;
  p.G = G;
  p.log2_g = G == 8 ? 3 : G == 4 ? 2 : G == 2 ? 1 : 0;
  p.S = S;
  p.W = W;
  p.prefix_blk = Pb;
  p.n_cta = n * G <= kRows ? 1 : 2;
  const int unit_rows = kRows * p.n_cta;
  p.n_grp = n < 2 || Pb == 0 ? 0 : (n * G + unit_rows - 1) / unit_rows;
  p.first_blk = p.n_grp > 0 ? Pb : 0;
  p.tiles_head = 0;
  const int per = unit_rows / G;  // sequences per group
  for (int j = 0; j < p.n_grp; ++j) {
    int lo = Pb;
    for (int s = j * per; s < std::min(n, (j + 1) * per); ++s) lo = std::min(lo, shared_win_lo(seqs[s0 + s].n_ctx, W));
    ShGroup& g = t.grp[j];
    g.x0 = p.tiles_head;
    g.lo = lo;
    g.sink = W > 0 ? std::min(S, lo) : 0;
    g.n_blk = g.sink + Pb - lo;
    p.tiles_head += (g.n_blk + kTileBlocks - 1) / kTileBlocks;
  }
  // at most 16 groups of 2^23 tiles: no overflow before the test
  if ((long long)HKV * p.tiles_head >= (1ll << 30)) return PA_EINVAL;
  // Blocks of the per-sequence pass, and its CTAs for a chunk size.
  long long own = 0;
  auto count_own = [&] {
    own = 0;
    for (int s = 0; s < n; ++s) {
      const pa_seq& q = seqs[s0 + s];
      const int lo = shared_win_lo(q.n_ctx, W), own_n = shared_own(q.n_ctx, lo, p.first_blk, S, W).n;
      t.s[s] = make_int4(q.q_off, q.n_ctx, own_n, lo);  // .z: the blocks until the chunks are counted
      own += own_n;
    }
  };
  count_own();
  auto own_ctas = [&](int chunk) {
    long long c = 0;
    for (int s = 0; s < n; ++s) c += (t.s[s].z + chunk - 1) / chunk;
    return c * HKV;
  };
  auto own_chunk = [&](int slots) {  // the smallest of 4, 8, ... 128 whose CTAs fit one wave of `slots`
    const long long even = (own * HKV + slots - 1) / slots;
    int c = (int)std::min<long long>(128, (std::max(4ll, even) + 3) / 4 * 4);
    for (long long k; c < 128 && (k = own_ctas(c)) > slots && k > (long long)n * HKV;) c = std::min(128, c + c / 8 / 4 * 4 + 4);
    return c;
  };
  // The prefix pass's units.  Both passes can run at once: the units left out
  // leave their SMs to the per-sequence pass, whose CTAs otherwise start when the
  // prefix pass ends.  Of a few numbers of units the one that ends first.
  const int T = HKV * p.tiles_head, max_units = std::min(kShUnits, std::max(1, n_sm / p.n_cta)), J = HKV * p.n_grp;
  const ShCost& cost = kShCost[p.n_cta - 1];
  p.n_units = 0;
  p.merge_ways = 0;
  int nt[8 * kShGroups], units = max_units;
  if (T > 0) {
    for (int j = 0; j < J; ++j) nt[j] = (t.grp[j % p.n_grp].n_blk + kTileBlocks - 1) / kTileBlocks;
    double best = 1e30;
    const double own_blk = (double)own * HKV, least_ctas = (double)n * HKV;
    for (int left = 0; left < max_units; left += 8 / p.n_cta) {
      const int use = std::min(max_units - left, T), free_sm = n_sm - p.n_cta * use;
      // a unit's cost when all are equal: its tiles, and its share of the groups' changes
      const int budget = (T + kShSegCost * std::max(0, J - use) + use - 1) / use + (J > 1 && J < use && use % J ? 1 : 0);
      const double prefix_us =
          cost.unit + (cost.tile * std::min(budget, 10) + cost.late * std::max(0, budget - 10)) * (W > 0 ? kShMaskedTile : 1.0);
      const double slots = kShOwnPerSm * free_sm, ctas = std::max(least_ctas, std::min(own_blk / 4, kShOwnWaves * slots));
      const double own_us = (kShOwnBlockUs * own_blk + kShOwnCtaUs * ctas) / (least_ctas > slots ? kShOwnFull : 1.0);
      // SM time before the prefix pass ends: that of the SMs left out; if none is, of the units with a tile less
      const double idle = free_sm > 1 ? free_sm * std::max(0.0, prefix_us - kShOwnStartUs)
                                      : p.n_cta * cost.late * std::max(0, budget * use - T);
      const double rest = std::max(0.0, own_us - idle);
      const double end = prefix_us + (rest > 0.0 ? rest / n_sm + cost.tail : 0.0);
      if (end < best) {
        best = end;
        units = use;
      }
      if (rest <= 0.0) break;  // fewer units only make the prefix pass longer
    }
    // With few sequences or a short prefix it is quicker that each reads the prefix too.
    double again = 0.0;
    for (int s = 0; s < n; ++s) again += (double)HKV * t.grp[s / per].n_blk;
    const double each = kShOwnStartUs + (kShOwnBlockUs * own_blk + kShAgainBlockUs * again) / n_sm;
    if (prefix_pass < 0 ? each < best : prefix_pass == 0) {
      p.n_grp = p.tiles_head = p.first_blk = 0;
      count_own();
    }
  }
  {  // Two waves keep the SMs full beside a prefix pass (48 sequences, windowed, 12104 blocks: 33.4 us, with one 37.3);
    // alone one is quicker (40 sequences, 16408 blocks: 29.5 us, with two 32.1).
    const int free_sm = p.tiles_head > 0 ? n_sm - p.n_cta * units : n_sm, wave = kShOwnPerSm * (free_sm > 0 ? free_sm : n_sm);
    p.chunk = own_chunk(wave * std::max(p.tiles_head > 0 ? kShOwnWaves : 1, (n * HKV + n * HKV / 4) / wave));
  }
  if (p.tiles_head > 0) {
    int budget = (T + units - 1) / units;
    while (!shared_pack(nt, J, budget, units, t.cut, p.n_units)) ++budget;
    int x = 0, c = 0, most = 0;
    for (int j = 0; j < J; ++j) {
      while (c + 1 < p.n_units && t.cut[c + 1] <= x) ++c;
      t.first_unit[j] = (uint8_t)c;
      x += nt[j];
      int e = c;
      while (e + 1 < p.n_units && t.cut[e + 1] < x) ++e;
      t.last_unit[j] = (uint8_t)e;
      most = std::max(most, e - c + 1);
    }
    p.merge_ways = most;
  }
  int chunks = 0, most = 0;
  for (int s = 0; s < n; ++s) {
    const int c = (t.s[s].z + p.chunk - 1) / p.chunk;
    t.s[s].z = chunks;
    for (int i = HKV * chunks; i < HKV * (chunks + c) && i < kShOwnListed; ++i) t.own_seq[i] = (uint16_t)s;
    chunks += c;
    most = std::max(most, c);
  }
  // Where every row is one CTA's there is nothing to merge.  (A merge by a row's last CTA in place of the kernel
  // saves a launch but takes longer: 3 sequences on 1024 tokens, 17 chunks a row, 8.9 us instead of 5.8.)
  p.merge_ways = p.tiles_head == 0 && most == 1 ? 0 : std::min(16, (p.merge_ways + most + 3) / 4);
  p.chunks_head = chunks;
  return PA_OK;
}

constexpr size_t kOwnPartial = (size_t)kHeadDim * 8 * sizeof(float), kOwnStats = 8 * sizeof(float2);
size_t pre_rows(const SharedParams& p) {  // of the partials
  return p.tiles_head > 0 ? ((size_t)p.n_units + (size_t)p.n_grp * p.HKV) * p.n_cta * kRows : 0;
}
size_t own_partials(const SharedParams& p) { return (size_t)p.HKV * p.chunks_head; }

}  // namespace

int pa_decode_shared(pa_handle h, int n_seq, const pa_seq* seqs, int n_prefix, int n_rows, const void* q,
                     const int8_t* k_pool, const int8_t* v_pool, const float* k_scale, const float* v_scale, const int32_t* block_table,
                     int n_sink_blk, int n_win_blk, float sm_scale, void* out, void* stream) {
  int rc = check_inputs(h, q, k_pool, v_pool, k_scale, v_scale, block_table, out);
  if (rc) return rc;
  if ((rc = decode_shared_check(h->HQ, h->HKV, h->max_pages, n_seq, seqs, n_prefix, n_sink_blk, sm_scale))) return rc;
  for (int s = 0; s < n_seq; ++s)
    if (seqs[s].q_off >= n_rows) return PA_EINVAL;
  const size_t row_bytes = (size_t)h->HQ * kHeadDim * sizeof(__nv_bfloat16);
  if (out != q && span_of(out, n_rows * row_bytes).meets(span_of(q, n_rows * row_bytes))) return PA_EINVAL;
  OnDevice dev(h->device);
  if (!dev.ok) return PA_ECUDA;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaStreamCaptureStatus capture = cudaStreamCaptureStatusNone;
  PA_CUDA(cudaStreamIsCapturing(st, &capture));
  SharedParams p{};
  SharedSeqs t;
  size_t pre = 0, own = 0;
  for (int s0 = 0; s0 < n_seq; s0 += kShSeqs) {
    if ((rc = decode_shared_plan(h->HQ, h->HKV, h->n_sm, seqs, s0, std::min(kShSeqs, n_seq - s0), n_prefix, n_sink_blk,
                                 n_win_blk, h->sh_pass, p, t)))
      return rc;
    pre = std::max(pre, pre_rows(p));
    own = std::max(own, own_partials(p));
  }
  DecodeMaps maps;
  if ((rc = pool_maps(h, k_pool, v_pool, maps))) return rc;
  const bool capturing = capture != cudaStreamCaptureStatusNone;
  if ((rc = reserve(h->sh_pre, pre * (kHeadDim * sizeof(float) + sizeof(float2)), capturing))) return rc;
  if ((rc = reserve(h->sh_own, own * (kOwnPartial + kOwnStats), capturing))) return rc;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.out = static_cast<__nv_bfloat16*>(out);
  p.k_pool = k_pool;
  p.v_pool = v_pool;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.block_table = block_table;
  p.bt_stride = h->max_pages;
  p.n_pool = h->n_pool;
  p.sm_scale_log2 = sm_scale * 1.4426950408889634f;
  p.pre_o = static_cast<float4*>(h->sh_pre.p);
  p.pre_ml = reinterpret_cast<float2*>(static_cast<char*>(h->sh_pre.p) + pre * kHeadDim * sizeof(float));
  p.own_o = static_cast<float4*>(h->sh_own.p);
  p.own_ml = reinterpret_cast<float2*>(static_cast<char*>(h->sh_own.p) + own * kOwnPartial);
  p.err = h->d_err;
  p.wait_ns = (unsigned long long)h->opt.wait_timeout_ms * 1000000ull;
  for (int s0 = 0; s0 < n_seq; s0 += kShSeqs) {
    if (n_seq > kShSeqs)
      (void)decode_shared_plan(h->HQ, h->HKV, h->n_sm, seqs, s0, std::min(kShSeqs, n_seq - s0), n_prefix, n_sink_blk,
                               n_win_blk, h->sh_pass, p, t);
    PA_CUDA(launch_decode_shared(p, t, maps, st));
  }
  return PA_OK;
}

int pa_debug_decode_shared_pass(pa_handle h, int prefix_pass) {
  if (!h || prefix_pass < -1 || prefix_pass > 1) return PA_EINVAL;
  h->sh_pass = prefix_pass;
  return PA_OK;
}

int pa_decode_shared_plan(int n_q_heads, int n_kv_heads, int max_pages_per_seq, int n_sm, int n_seq,
                          const pa_seq* seqs, int n_prefix, int n_sink_blk, int n_win_blk, int prefix_pass,
                          int32_t* prefix_out, int prefix_cap, int* n_prefix_runs, int32_t* own_out, int own_cap,
                          int* n_own_runs) {
  if (n_sm < 1 || prefix_pass < -1 || prefix_pass > 1 || max_pages_per_seq < 1 || !n_prefix_runs || !n_own_runs) return PA_EINVAL;
  int rc = decode_shared_check(n_q_heads, n_kv_heads, max_pages_per_seq, n_seq, seqs, n_prefix, n_sink_blk, 1.f);
  if (rc) return rc;
  SharedParams p{};
  SharedSeqs t;
  if ((rc = decode_shared_plan(n_q_heads, n_kv_heads, n_sm, seqs, 0, std::min(n_seq, kShSeqs), n_prefix, n_sink_blk,
                               n_win_blk, prefix_pass, p, t)))
    return rc;
  const int per = kRows * p.n_cta / p.G;
  int np = 0;
  for (int g = 0; g < p.HKV; ++g)
    for (int j = 0; j < p.n_grp; ++j) {
      const ShGroup& gr = t.grp[j];
      const int nt = (gr.n_blk + kTileBlocks - 1) / kTileBlocks;
      const int a = g * p.tiles_head + gr.x0;
      for (int t0 = 0; t0 < nt;) {
        const int c = (int)(std::upper_bound(t.cut, t.cut + p.n_units, a + t0) - t.cut) - 1;
        const int t1 = std::min(nt, t.cut[c + 1] - a);
        if (prefix_out) {
          if (np >= prefix_cap) return PA_EINVAL;
          int32_t* o = prefix_out + 8 * np;
          o[0] = c;
          o[1] = g;
          o[2] = j * per;
          o[3] = std::min(p.n_seq, (j + 1) * per) - o[2];
          o[4] = gr.sink;
          o[5] = gr.lo;
          o[6] = t0 * kTileBlocks;
          o[7] = std::min(gr.n_blk, t1 * kTileBlocks);
        }
        ++np;
        t0 = t1;
      }
    }
  int no = 0;
  for (int s = 0; s < p.n_seq; ++s) {
    const ShOwn o = shared_own(t.s[s].y, t.s[s].w, p.first_blk, p.S, p.W);
    const int n_ch = (o.n + p.chunk - 1) / p.chunk;
    for (int c = 0; c < n_ch; ++c)
      for (int g = 0; g < p.HKV; ++g) {
        if (own_out) {
          if (no >= own_cap) return PA_EINVAL;
          int32_t* r = own_out + 7 * no;
          r[0] = s;
          r[1] = g;
          r[2] = p.first_blk;
          r[3] = o.sink;
          r[4] = o.lo;
          r[5] = c * p.chunk;
          r[6] = std::min(o.n, (c + 1) * p.chunk);
        }
        ++no;
      }
  }
  *n_prefix_runs = np;
  *n_own_runs = no;
  return PA_OK;
}

int pa_debug_maskset(pa_handle h, int n_seq, const pa_seq* seqs, int n_sink_blk, int n_win_blk,
                     int32_t* row_counts, int32_t* unit_blocks, int cap, int32_t* units_out, int units_cap,
                     int* n_units, void* stream) {
  if (!h || !row_counts || !unit_blocks || !units_out || !n_units || cap <= 0) return PA_EINVAL;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  int rc = prepare(h, n_seq, seqs, n_sink_blk, n_win_blk, st);
  if (rc) return rc;
  const Plan& P = h->plan;
  *n_units = (int)P.units.size();
  if ((int)P.units.size() > units_cap) return PA_EINVAL;
  for (size_t i = 0; i < P.units.size(); ++i) {
    units_out[4 * i + 0] = P.units[i].seq;
    units_out[4 * i + 1] = P.units[i].g;
    units_out[4 * i + 2] = P.units[i].t0;
    units_out[4 * i + 3] = P.units[i].n_tiles;
  }
  PA_CUDA(launch_debug_maskset(h->d_seqs, h->d_units, (int)P.units.size(), 2 * h->TQ, h->G, n_sink_blk, n_win_blk,
                               row_counts, unit_blocks, cap, st));
  return pa_last_error(h, stream);
}

}  // extern "C"

// ======================================================================
// The 4-bit pool and the page operators.
// ======================================================================
namespace {
// No C++ exception leaves a C entry point.
template <typename F>
int guarded(F f) {
  try {
    return f();
  } catch (const std::bad_alloc&) {
    return PA_ENOMEM;
  } catch (...) {
    return PA_EINVAL;
  }
}

struct Shape4 {
  int HQ, HKV, n_pool, max_pages;
};
Shape4 shape_of(pa_handle h) { return Shape4{h->HQ, h->HKV, h->n_pool, h->max_pages}; }
bool shape_ok(const Shape4& d) { return heads_ok(d.HQ, d.HKV) && d.n_pool > 0 && d.max_pages > 0; }
Span pool4_span(const Shape4& d, const void* pool) { return span_of(pool, (size_t)d.n_pool * d.HKV * kT4Bytes); }
Span table_span(const int32_t* bt, int rows, int max_pages) { return span_of(bt, (size_t)rows * max_pages * sizeof(int32_t)); }

// Sequences with new or wanted tokens [q_start, q_start + n_q): checks, and the rows their arrays need.
int token_seqs(const Shape4& d, int n_seq, const pa_seq* seqs, long long& rows) {
  if (!seqs) return PA_EINVAL;
  rows = 0;
  for (int s = 0; s < n_seq; ++s) {
    const pa_seq& a = seqs[s];
    if (a.n_q < 1 || a.q_start < 0 || a.q_off < 0 || (long long)a.q_start + a.n_q > a.n_ctx ||
        (long long)a.q_start + a.n_q > (long long)d.max_pages * kPage || (long long)a.q_off + a.n_q > (1ll << 30))
      return PA_EINVAL;
    rows = std::max(rows, (long long)a.q_off + a.n_q);
  }
  return rows_shared(n_seq, seqs) ? PA_EINVAL : PA_OK;
}

int kv4_append_args(const Shape4& d, int n_seq, const pa_seq* seqs, const pa_rows* k, const pa_rows* v,
                    const int32_t* bt, uint8_t* pool, Kv4RowsParams& p) {
  if (!k || !v || !bt || !pool || !aligned(bt, 4) || !aligned(pool, 16)) return PA_EINVAL;
  long long rows;
  const int rc = token_seqs(d, n_seq, seqs, rows);
  if (rc) return rc;
  Span ks, vs;
  if (!rows_ok(k, rows, d.HKV, p.k, ks) || !rows_ok(v, rows, d.HKV, p.v, vs)) return PA_EINVAL;
  const Span w = pool4_span(d, pool);
  if (w.meets(ks) || w.meets(vs) || w.meets(table_span(bt, n_seq, d.max_pages))) return PA_EINVAL;
  p.pool = pool;
  return PA_OK;
}

int kv4_gather_args(const Shape4& d, int n_seq, const pa_seq* seqs, const int32_t* bt, const uint8_t* pool, int n_rows,
                    void* k_out, void* v_out, Kv4RowsParams& p) {
  if (!bt || !pool || !aligned(bt, 4) || !aligned(pool, 16) || (!k_out && !v_out)) return PA_EINVAL;
  if (!aligned(k_out, 16) || !aligned(v_out, 16)) return PA_EINVAL;
  long long rows;
  const int rc = token_seqs(d, n_seq, seqs, rows);
  if (rc) return rc;
  if (rows > n_rows) return PA_EINVAL;
  const size_t bytes = (size_t)n_rows * d.HKV * kHeadDim * 2;
  const Span ko = span_of(k_out, k_out ? bytes : 0), vo = span_of(v_out, v_out ? bytes : 0);
  for (const Span& in : {pool4_span(d, pool), table_span(bt, n_seq, d.max_pages)})
    if ((k_out && ko.meets(in)) || (v_out && vo.meets(in))) return PA_EINVAL;
  if (k_out && v_out && ko.meets(vo)) return PA_EINVAL;
  p.k_out = static_cast<__nv_bfloat16*>(k_out);
  p.v_out = static_cast<__nv_bfloat16*>(v_out);
  p.pool = const_cast<uint8_t*>(pool);  // only read
  return PA_OK;
}

int kv4_attention_args(bool decode, const Shape4& d, int n_seq, const pa_seq* seqs, int n_rows, const void* q,
                       const void* gate, const uint8_t* pool, const int32_t* bt, int S, float sm_scale, const void* out) {
  if (n_seq < 1 || !seqs || !q || !pool || !bt || !out || S < 0 || !std::isfinite(sm_scale) || sm_scale < 0.f)
    return PA_EINVAL;
  if (!aligned(q, 16) || !aligned(gate, 16) || !aligned(pool, 16) || !aligned(out, 16) || !aligned(bt, 4)) return PA_EINVAL;
  long long rows;
  const int rc = token_seqs(d, n_seq, seqs, rows);
  if (rc) return rc;
  if (rows > n_rows) return PA_EINVAL;
  for (int s = 0; s < n_seq; ++s) {
    if ((long long)seqs[s].n_ctx > std::min((long long)d.max_pages * kPage, 1ll << 30)) return PA_EINVAL;
    if (decode && !decode_seq_ok(seqs[s], d.max_pages)) return PA_EINVAL;
  }
  if (decode && d.HQ / d.HKV > 8) return PA_EINVAL;
  const size_t bytes = (size_t)n_rows * d.HQ * kHeadDim * 2;
  const Span o = span_of(out, bytes);
  if (o.meets(span_of(q, bytes)) && !(decode && out == q)) return PA_EINVAL;
  if (gate && o.meets(span_of(gate, bytes))) return PA_EINVAL;
  if (o.meets(pool4_span(d, pool)) || o.meets(table_span(bt, n_seq, d.max_pages))) return PA_EINVAL;
  return PA_OK;
}

// The pools of a call on pages, in the kernels' form; `spans`: the arrays that must lie apart, to which they are added.
int page_parts(int n_pool, int n_parts, const pa_part* parts, PageParts& out, std::vector<Span>& spans) {
  if (n_parts < 0 || n_parts > PA_MAX_PARTS || (n_parts > 0 && !parts)) return PA_EINVAL;
  out.n = n_parts;
  for (int i = 0; i < n_parts; ++i) {
    const pa_part& a = parts[i];
    if (!a.data || !aligned(a.data, 4) || a.page_bytes <= 0 || a.page_bytes % 4 || a.page_bytes > (1ll << 30)) return PA_EINVAL;
    out.part[i] = a;
    spans.push_back(span_of(a.data, (size_t)n_pool * (size_t)a.page_bytes));
  }
  std::sort(spans.begin(), spans.end(), [](const Span& a, const Span& b) { return a.lo < b.lo; });
  for (size_t i = 1; i < spans.size(); ++i)
    if (spans[i - 1].meets(spans[i])) return PA_EINVAL;
  return PA_OK;
}

// Whole numbers >= 0 told apart (open addressing, half full at most).
class Distinct {
 public:
  explicit Distinct(int n) {
    size_t size = 16;
    while (size < 2 * (size_t)n) size *= 2;
    slot_.assign(size, -1);
  }
  bool add(int x) { return find(x, true) < 0; }  // whether it is new
  bool has(int x) { return find(x, false) >= 0; }

 private:
  int find(int x, bool put) {
    size_t i = (size_t)((uint32_t)x * 2654435769u) & (slot_.size() - 1);
    for (; slot_[i] >= 0; i = (i + 1) & (slot_.size() - 1))
      if (slot_[i] == x) return x;
    if (put) slot_[i] = x;
    return -1;
  }
  std::vector<int> slot_;
};

int fork_args(int n_pool, int max_pages, int n_fork, const pa_fork* forks, int n_rows, int32_t* bt, int n_parts,
              const pa_part* parts, PageParts& out) {
  if (!forks || !bt || !aligned(bt, 4) || n_rows < 1) return PA_EINVAL;
  Distinct dst(n_fork), page(n_fork);
  for (int i = 0; i < n_fork; ++i) {
    const pa_fork& f = forks[i];
    if (f.src_row < 0 || f.src_row >= n_rows || f.dst_row < 0 || f.dst_row >= n_rows || f.n_tok < 0 ||
        f.n_tok > std::min((long long)max_pages * kPage, 1ll << 30) || !dst.add(f.dst_row))
      return PA_EINVAL;
    if (f.n_tok % kPage && (f.new_page < 0 || f.new_page >= n_pool || !page.add(f.new_page))) return PA_EINVAL;
  }
  for (int i = 0; i < n_fork; ++i)
    if (dst.has(forks[i].src_row)) return PA_EINVAL;
  std::vector<Span> spans{table_span(bt, n_rows, max_pages)};
  return page_parts(n_pool, n_parts, parts, out, spans);
}

int compact_args(int n_pool, int max_pages, int n_seq, const pa_seq* seqs, int S, const int32_t* bt, int32_t* nt,
                 int n_parts, const pa_part* parts, int32_t* n_live, PageParts& out) {
  if (n_seq < 0 || (n_seq > 0 && (!seqs || !bt || !nt)) || S < 0 || !n_live || !aligned(n_live, 4)) return PA_EINVAL;
  if (n_pool > (1 << 30)) return PA_EINVAL;  // the kernels' page numbers, rounded up to words of marks, are ints
  if (!aligned(bt, 4) || !aligned(nt, 4)) return PA_EINVAL;
  for (int s = 0; s < n_seq; ++s)
    if (seqs[s].n_ctx < 0 || seqs[s].n_ctx > (long long)max_pages * kPage || seqs[s].n_ctx > (1 << 30)) return PA_EINVAL;
  std::vector<Span> spans{span_of(n_live, sizeof(int32_t))};
  if (n_seq > 0) {
    spans.push_back(table_span(bt, n_seq, max_pages));
    if (nt != bt) spans.push_back(table_span(nt, n_seq, max_pages));
  }
  return page_parts(n_pool, n_parts, parts, out, spans);
}

int is_capturing(cudaStream_t st, bool& capturing) {
  cudaStreamCaptureStatus c = cudaStreamCaptureStatusNone;
  PA_CUDA(cudaStreamIsCapturing(st, &c));
  capturing = c != cudaStreamCaptureStatusNone;
  return PA_OK;
}

// The launches of an append or a gather: up to kQkvSeqs sequences each.
template <typename F>
int kv4_rows(pa_handle h, Kv4RowsParams& p, int n_seq, const pa_seq* seqs, const int32_t* bt, F launch) {
  p.block_table = bt;
  p.bt_stride = h->max_pages;
  p.n_pool = h->n_pool;
  p.HKV = h->HKV;
  p.err = h->d_err;
  OnDevice dev(h->device);
  if (!dev.ok) return PA_ECUDA;
  QkvSeqs<kQkvSeqs> tab;
  for (int s0 = 0; s0 < n_seq; s0 += kQkvSeqs) {
    const int n = std::min(kQkvSeqs, n_seq - s0);
    int first = 0;
    p.same_len = seqs[s0].n_q;
    for (int i = 0; i < n; ++i) {
      const pa_seq& a = seqs[s0 + i];
      tab.s[i] = make_int4(a.q_off, a.q_start, first, 0);
      first += a.n_q;  // at most 2^30: the sequences' rows are disjoint
      if (a.n_q != p.same_len) p.same_len = 0;
    }
    p.n_seq = n;
    p.n_tok = first;
    p.bt_row0 = s0;
    PA_CUDA(launch(p, tab));
  }
  return PA_OK;
}

// A launch of the 4-bit decode: sequences [s0, s0 + n) -> its table and split: runs of at most T blocks, with the least T
// whose runs are as many as the GPU's warps, or that many more than the pairs where those alone fill the warps (the CTAs
// over one wave start as others end).  T is at least kK4LeastBlocks, so that few keys are not spread over more
// partials than their merge is worth.
constexpr long long kK4LeastBlocks = 2;
int kv4_decode_plan(pa_handle h, const pa_seq* seqs, int s0, int n, int S, int W, Kv4DecodeParams& p, Kv4DecodeSeqs& tab) {
  const long long HKV = h->HKV, cta = kv4_decode_cta_warps(), warps = kv4_decode_warps(h->n_sm);
  long long most = 1, total = 0;
  int len[kKv4Seqs];
  for (int i = 0; i < n; ++i) {
    len[i] = decode_n_vis(seqs[s0 + i].n_ctx, S, W);
    most = std::max(most, (long long)len[i]);
    total += HKV * len[i];
  }
  if (total >= (1ll << 30)) return PA_EINVAL;
  const long long room = std::min(kKv4Ctas * cta, 2 * n * HKV <= warps ? warps : warps + n * HKV);
  const auto runs_of = [&](long long T) {
    long long r = 0;
    for (int i = 0; i < n; ++i) r += (len[i] + T - 1) / T;
    return HKV * r;
  };
  long long lo = std::max(kK4LeastBlocks, total / room), hi = std::max(lo, most);  // T = most: a run each, at most 512 x 8
  while (lo < hi) {
    const long long mid = (lo + hi) / 2;
    if (runs_of(mid) <= room) hi = mid;
    else lo = mid + 1;
  }
  p.n_seq = n;
  p.bt_row0 = s0;
  p.most_runs = 1;
  // runs that are still to be had go to the sequences whose runs are the longest, one more for each of their pairs
  long long first = 0, left = room - runs_of(lo);
  for (int i = 0; i < n; ++i) {
    int r = (int)((len[i] + lo - 1) / lo);
    if (left >= HKV && lo > kK4LeastBlocks && (len[i] + lo - 2) / (lo - 1) > r) {
      ++r;
      left -= HKV;
    }
    tab.seq[i] = make_int4(seqs[s0 + i].q_off, seqs[s0 + i].n_ctx, (int)first, r);
    for (long long c = (first + cta - 1) / cta; c * cta < first + r * HKV; ++c) tab.cta_seq[c] = (uint16_t)i;
    first += r * HKV;
    p.most_runs = std::max(p.most_runs, r);
  }
  p.n_runs = (int)first;
  return PA_OK;
}

int kv4_decode(pa_handle h, int n_seq, const pa_seq* seqs, const void* q, const uint8_t* pool, const int32_t* bt, int S,
               int W, float sm_scale, void* out, cudaStream_t st) {
  OnDevice dev(h->device);
  if (!dev.ok) return PA_ECUDA;
  Kv4DecodeParams p{};
  Kv4DecodeSeqs tab;
  size_t parts = 0;
  int rc;
  for (int s0 = 0; s0 < n_seq; s0 += kKv4Seqs) {
    const int n = std::min(kKv4Seqs, n_seq - s0);
    if ((rc = kv4_decode_plan(h, seqs, s0, n, S, W, p, tab))) return rc;
    if (p.most_runs > 1) parts = std::max(parts, (size_t)p.n_runs);
  }
  const size_t o_bytes = parts * kKv4Part * sizeof(float4), need = o_bytes + parts * 8 * sizeof(float2);
  if (h->k4_part.bytes < need) {
    bool capturing;
    if ((rc = is_capturing(st, capturing)) || (rc = reserve(h->k4_part, need, capturing))) return rc;
  }
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.out = static_cast<__nv_bfloat16*>(out);
  p.pool = pool;
  p.block_table = bt;
  p.bt_stride = h->max_pages;
  p.n_pool = h->n_pool;
  p.S = S;
  p.W = W;
  p.HQ = h->HQ;
  p.HKV = h->HKV;
  p.G = h->G;
  p.sm_scale_log2 = sm_scale * 1.4426950408889634f;
  p.part = static_cast<float*>(h->k4_part.p);
  p.nw = reinterpret_cast<float2*>(static_cast<char*>(h->k4_part.p) + o_bytes);
  p.err = h->d_err;
  p.wait_ns = (unsigned long long)h->opt.wait_timeout_ms * 1000000ull;
  for (int s0 = 0; s0 < n_seq; s0 += kKv4Seqs) {
    if (n_seq > kKv4Seqs) (void)kv4_decode_plan(h, seqs, s0, std::min(kKv4Seqs, n_seq - s0), S, W, p, tab);
    PA_CUDA(launch_kv4_decode(p, tab, st));
  }
  return PA_OK;
}

int compact(pa_handle h, int n_seq, const pa_seq* seqs, int S, int W, const int32_t* bt, int32_t* nt,
            const PageParts& parts, int32_t* n_live, cudaStream_t st) {
  OnDevice dev(h->device);
  if (!dev.ok) return PA_ECUDA;
  if (n_seq == 0) {
    PA_CUDA(cudaMemsetAsync(n_live, 0, sizeof(int32_t), st));
    return PA_OK;
  }
  bool capturing;
  int rc = is_capturing(st, capturing);
  if (rc) return rc;
  const size_t n = (size_t)h->n_pool, live_bytes = (n + 31) / 32 * sizeof(uint32_t);
  const size_t moves_at = (2 * sizeof(int) + live_bytes + 15) / 16 * 16;
  if ((rc = reserve(h->pages, moves_at + n * (sizeof(PageMove) + sizeof(int32_t)), capturing))) return rc;
  char* ws = static_cast<char*>(h->pages.p);
  CompactParams p{};
  Contexts ctx;
  p.S = S;
  p.W = W;
  p.table = bt;
  p.new_table = nt;
  p.stride = h->max_pages;
  p.n_pool = h->n_pool;
  p.count = reinterpret_cast<int*>(ws);
  p.live = reinterpret_cast<uint32_t*>(ws + 2 * sizeof(int));
  p.moves = reinterpret_cast<PageMove*>(ws + moves_at);
  p.moved_to = reinterpret_cast<int32_t*>(ws + moves_at + n * sizeof(PageMove));
  p.n_live = n_live;
  p.err = h->d_err;
  auto take = [&](int s0) {
    p.row0 = s0;
    p.n_seq = std::min(kPageRows, n_seq - s0);
    for (int i = 0; i < p.n_seq; ++i) ctx.n_ctx[i] = seqs[s0 + i].n_ctx;
  };
  long long entries = 0;  // in use
  for (int s = 0; s < n_seq; ++s) entries += decode_n_vis(seqs[s].n_ctx + 1, S, W);
  if (n_seq <= kPageRows && entries <= kOneCtaEntries && h->n_pool <= kOneCtaPages) {
    take(0);
    PA_CUDA(launch_pages_mark_plan(p, ctx, st));
  } else {
    PA_CUDA(cudaMemsetAsync(p.live, 0, live_bytes, st));
    for (int s0 = 0; s0 < n_seq; s0 += kPageRows) {
      take(s0);
      PA_CUDA(launch_pages_mark(p, ctx, st));
    }
    PA_CUDA(launch_pages_plan(p, st));
  }
  PageParts none;
  none.n = 0;
  for (int s0 = 0; s0 < n_seq; s0 += kPageRows) {
    take(s0);
    PA_CUDA(launch_pages_apply(p, ctx, s0 == 0 ? parts : none, h->n_sm, st));
  }
  return PA_OK;
}
}  // namespace

extern "C" {

int pa_kv4_append(pa_handle h, int n_seq, const pa_seq* seqs, const pa_rows* k, const pa_rows* v,
                  const int32_t* block_table, uint8_t* pool, void* stream) {
  if (!h || n_seq < 0) return PA_EINVAL;
  if (n_seq == 0) return PA_OK;
  return guarded([&] {
    Kv4RowsParams p{};
    const int rc = kv4_append_args(shape_of(h), n_seq, seqs, k, v, block_table, pool, p);
    return rc ? rc : kv4_rows(h, p, n_seq, seqs, block_table, [&](const Kv4RowsParams& a, const QkvSeqs<kQkvSeqs>& t) {
      return launch_kv4_append(a, t, static_cast<cudaStream_t>(stream));
    });
  });
}

int pa_kv4_gather(pa_handle h, int n_seq, const pa_seq* seqs, const int32_t* block_table, const uint8_t* pool,
                  int n_rows, void* k_out, void* v_out, void* stream) {
  if (!h || n_seq < 0) return PA_EINVAL;
  if (n_seq == 0) return PA_OK;
  return guarded([&] {
    Kv4RowsParams p{};
    const int rc = kv4_gather_args(shape_of(h), n_seq, seqs, block_table, pool, n_rows, k_out, v_out, p);
    return rc ? rc : kv4_rows(h, p, n_seq, seqs, block_table, [&](const Kv4RowsParams& a, const QkvSeqs<kQkvSeqs>& t) {
      return launch_kv4_gather(a, t, static_cast<cudaStream_t>(stream));
    });
  });
}

int pa_kv4_decode(pa_handle h, int n_seq, const pa_seq* seqs, int n_rows, const void* q, const uint8_t* pool,
                  const int32_t* block_table, int n_sink_blk, int n_win_blk, float sm_scale, void* out, void* stream) {
  if (!h) return PA_EINVAL;
  return guarded([&] {
    const int rc = kv4_attention_args(true, shape_of(h), n_seq, seqs, n_rows, q, nullptr, pool, block_table, n_sink_blk,
                                      sm_scale, out);
    return rc ? rc : kv4_decode(h, n_seq, seqs, q, pool, block_table, n_sink_blk, n_win_blk, sm_scale, out,
                                static_cast<cudaStream_t>(stream));
  });
}

int pa_kv4_prefill(pa_handle h, int n_seq, const pa_seq* seqs, int n_rows, const void* q, const void* q_gate,
                   const uint8_t* pool, const int32_t* block_table, int n_sink_blk, int n_win_blk, float sm_scale,
                   void* out, void* stream) {
  if (!h) return PA_EINVAL;
  return guarded([&] {
    int rc = kv4_attention_args(false, shape_of(h), n_seq, seqs, n_rows, q, q_gate, pool, block_table, n_sink_blk,
                                sm_scale, out);
    if (rc) return rc;
    OnDevice dev(h->device);
    if (!dev.ok) return PA_ECUDA;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    bool capturing;
    if ((rc = is_capturing(st, capturing))) return rc;
    if (capturing) return PA_EINVAL;  // the plan on the device is the last call's
    if ((rc = prepare(h, n_seq, seqs, n_sink_blk, n_win_blk, st, true))) return rc;
    return launch_plan(h, h->plan, h->d_seqs, h->d_units, n_seq, q, nullptr, nullptr, nullptr, nullptr, block_table,
                       n_sink_blk, n_win_blk, sm_scale, out, st, q_gate, pool);
  });
}

int pa_pages_fork(pa_handle h, int n_fork, const pa_fork* forks, int n_rows, int32_t* block_table, int n_parts,
                  const pa_part* parts, void* stream) {
  if (!h || n_fork < 0) return PA_EINVAL;
  if (n_fork == 0) return PA_OK;
  return guarded([&]() -> int {
    PageParts in;
    const int rc = fork_args(h->n_pool, h->max_pages, n_fork, forks, n_rows, block_table, n_parts, parts, in);
    if (rc) return rc;
    OnDevice dev(h->device);
    if (!dev.ok) return PA_ECUDA;
    ForkParams p{};
    Forks t;
    p.table = block_table;
    p.stride = h->max_pages;
    p.n_pool = h->n_pool;
    p.err = h->d_err;
    for (int f0 = 0; f0 < n_fork; f0 += kPageRows) {
      p.n_fork = std::min(kPageRows, n_fork - f0);
      for (int i = 0; i < p.n_fork; ++i) {
        const pa_fork& f = forks[f0 + i];
        t.fork[i] = make_int4(f.src_row, f.dst_row, f.n_tok, f.new_page);
      }
      PA_CUDA(launch_pages_fork(p, t, in, h->n_sm, static_cast<cudaStream_t>(stream)));
    }
    return PA_OK;
  });
}

int pa_pages_compact(pa_handle h, int n_seq, const pa_seq* seqs, int n_sink_blk, int n_win_blk,
                     const int32_t* block_table, int32_t* new_table, int n_parts, const pa_part* parts,
                     int32_t* n_live, void* stream) {
  if (!h) return PA_EINVAL;
  return guarded([&] {
    PageParts in;
    const int rc = compact_args(h->n_pool, h->max_pages, n_seq, seqs, n_sink_blk, block_table, new_table, n_parts, parts,
                                n_live, in);
    return rc ? rc : compact(h, n_seq, seqs, n_sink_blk, n_win_blk, block_table, new_table, in, n_live,
                             static_cast<cudaStream_t>(stream));
  });
}

int pa_debug_kv4_append_check(int n_q_heads, int n_kv_heads, int n_pool_pages, int max_pages_per_seq, int n_seq,
                              const pa_seq* seqs, const pa_rows* k, const pa_rows* v, const int32_t* block_table,
                              uint8_t* pool) {
  const Shape4 d{n_q_heads, n_kv_heads, n_pool_pages, max_pages_per_seq};
  if (!shape_ok(d) || n_seq < 0) return PA_EINVAL;
  if (n_seq == 0) return PA_OK;
  return guarded([&] {
    Kv4RowsParams p{};
    return kv4_append_args(d, n_seq, seqs, k, v, block_table, pool, p);
  });
}

int pa_debug_kv4_gather_check(int n_q_heads, int n_kv_heads, int n_pool_pages, int max_pages_per_seq, int n_seq,
                              const pa_seq* seqs, const int32_t* block_table, const uint8_t* pool, int n_rows,
                              void* k_out, void* v_out) {
  const Shape4 d{n_q_heads, n_kv_heads, n_pool_pages, max_pages_per_seq};
  if (!shape_ok(d) || n_seq < 0) return PA_EINVAL;
  if (n_seq == 0) return PA_OK;
  return guarded([&] {
    Kv4RowsParams p{};
    return kv4_gather_args(d, n_seq, seqs, block_table, pool, n_rows, k_out, v_out, p);
  });
}

int pa_debug_kv4_attention_check(int decode, int n_q_heads, int n_kv_heads, int n_pool_pages, int max_pages_per_seq,
                                 int n_seq, const pa_seq* seqs, int n_rows, const void* q, const void* q_gate,
                                 const uint8_t* pool, const int32_t* block_table, int n_sink_blk, float sm_scale,
                                 void* out) {
  const Shape4 d{n_q_heads, n_kv_heads, n_pool_pages, max_pages_per_seq};
  if (!shape_ok(d) || (decode && q_gate)) return PA_EINVAL;
  return guarded([&] {
    return kv4_attention_args(decode != 0, d, n_seq, seqs, n_rows, q, q_gate, pool, block_table, n_sink_blk, sm_scale, out);
  });
}

int pa_debug_pages_fork_check(int n_pool_pages, int max_pages_per_seq, int n_fork, const pa_fork* forks, int n_rows,
                              int32_t* block_table, int n_parts, const pa_part* parts) {
  if (n_pool_pages <= 0 || max_pages_per_seq <= 0 || n_fork < 0) return PA_EINVAL;
  if (n_fork == 0) return PA_OK;
  return guarded([&] {
    PageParts in;
    return fork_args(n_pool_pages, max_pages_per_seq, n_fork, forks, n_rows, block_table, n_parts, parts, in);
  });
}

int pa_debug_pages_compact_check(int n_pool_pages, int max_pages_per_seq, int n_seq, const pa_seq* seqs,
                                 int n_sink_blk, const int32_t* block_table, int32_t* new_table, int n_parts,
                                 const pa_part* parts, int32_t* n_live) {
  if (n_pool_pages <= 0 || max_pages_per_seq <= 0) return PA_EINVAL;
  return guarded([&] {
    PageParts in;
    return compact_args(n_pool_pages, max_pages_per_seq, n_seq, seqs, n_sink_blk, block_table, new_table, n_parts, parts,
                        n_live, in);
  });
}

}  // extern "C"
