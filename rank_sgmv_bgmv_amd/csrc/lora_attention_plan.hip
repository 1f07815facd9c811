// The plan of an attention step: which rows read which key tiles, in pieces of
// about the same length, made once a step on the device by one workgroup and
// read by every layer's kernels.
//
// A sequence whose n * group rows (its queries times the query heads of a cache
// head) fit the kernel for few rows is one unit, others are units of many_rows
// rows.  With W key tiles in all units of a kind, a piece has max(least, W /
// target) tiles, so that a launch has about `target` of them for each cache head
// however few and long the sequences are; units are cut into equal pieces.
//
// One workgroup: 7 us for one sequence, 14 for 260, once a step for all layers.

#include "lora_device.hpp"
#include "lora_layer.hpp"

namespace lora {
namespace {

constexpr int kAttnPlanThreads = 256, kAttnPlanWaves = kAttnPlanThreads / 64;

// Sum over the workgroup of what lies before a thread, and of all (Op: the sum or the maximum).
template <typename T, typename Op>
__device__ __forceinline__ T block_scan(T v, T none, T *part, Op op, T *all) {
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  T inc = v;
#pragma unroll
  for (int o = 1; o < 64; o *= 2) {
    const T u = __shfl_up(inc, o);
    if (lane >= o) inc = op(inc, u);
  }
  __syncthreads();  // the last scan's parts were read
  if (lane == 63) part[wave] = inc;
  __syncthreads();
  T before = none, total = none;
#pragma unroll
  for (int w = 0; w < kAttnPlanWaves; ++w) {
    if (w == wave) before = total;
    total = op(total, part[w]);
  }
  const T ex = __shfl_up(inc, 1);
  *all = total;
  return lane ? op(before, ex) : before;
}
__device__ __forceinline__ int scan_sum(int v, int *part, int *all) {
  return block_scan(v, 0, part, [](int a, int b) { return a + b; }, all);
}

// The key tiles of rows row0 .. row0 + rows - 1 of a sequence.
__device__ inline void unit_tiles(const AttnPlanArgs &a, AttnUnit &u) {
  const int context = u.len - u.n, first = u.row0 / a.s.group, last = (u.row0 + u.rows - 1) / a.s.group;
  // the positions of the rows: drafted tokens stand anywhere from the context's end on, and see each other
  const int p_lo = a.tree ? context : context + first;
  const int hi = min(u.len, a.tree ? u.len : context + last + 1);
  const int lo = a.window ? max(0, p_lo - a.window + 1) : 0;
  if (hi <= 0) {
    u.ntiles = u.sink_tiles = u.main = 0;
    return;
  }
  u.main = min(lo, hi) / kKeyTile;
  u.sink_tiles = a.window ? min((min(a.sinks, hi) + kKeyTile - 1) / kKeyTile, u.main) : 0;
  u.ntiles = u.sink_tiles + (hi + kKeyTile - 1) / kKeyTile - u.main;
}

__device__ __forceinline__ void put_unit(char *at, const AttnUnit &u) {
  const int4 w[4] = {make_int4(u.q0, u.n, u.len, u.row0), make_int4(u.rows, u.seq, u.ntiles, u.sink_tiles),
                     make_int4(u.main, u.nsplit, u.slot, 0), make_int4(0, 0, 0, 0)};
#pragma unroll
  for (int i = 0; i < 4; ++i) gstore(at + 16 * i, w[i]);
}

__global__ __launch_bounds__(kAttnPlanThreads) void attention_plan_kernel(AttnPlanArgs a) {
  __shared__ int part[kAttnPlanWaves];
  __shared__ int64_t part64[kAttnPlanWaves];
  const AttnShape &s = a.s;
  const int tid = threadIdx.x;
  char *base = reinterpret_cast<char *>(a.plan);
  int *toff = reinterpret_cast<int *>(base + s.toff);
  int errors = 0, seen = 0;  // seen: the largest offset so far
  int n_units[ATTN_KINDS] = {0, 0};
  int64_t tiles[ATTN_KINDS] = {0, 0};

  // sequences: which kind, how many units; the units of few rows are made here
  for (int s0 = 0; s0 < s.S; s0 += kAttnPlanThreads) {
    const int q = s0 + tid;
    const bool live = q < s.S;
    const int lo = live ? gload<int>(a.q_off + q) : 0, hi = live ? gload<int>(a.q_off + q + 1) : 0;
    const int len = live ? gload<int>(a.lens + q) : 0;
    int top;
    const int before = block_scan(live ? max(lo, hi) : 0, 0, part, [](int x, int y) { return max(x, y); }, &top);
    const bool ok = live && lo >= max(before, seen) && hi >= lo && hi <= s.T && hi - lo <= a.max_q && len >= 0 &&
                    len <= a.capacity;
    seen = max(seen, top);
    if (live && !ok) ++errors;
    const int n = ok ? hi - lo : 0;
    const int rows = n * s.group;
    const bool few = n > 0 && rows <= s.few_rows;
    const int many = few || n == 0 ? 0 : (rows - 1) / s.many_rows + 1;
    int all;
    const int fu = scan_sum(few, part, &all) + n_units[ATTN_FEW];
    n_units[ATTN_FEW] += all;
    const int mu = scan_sum(many, part, &all) + n_units[ATTN_MANY];
    n_units[ATTN_MANY] += all;
    if (live) gstore(toff + q, mu);
    if (few) {
      AttnUnit u{lo, n, len, 0, rows, q, 0, 0, 0, 1, 0, {}};
      unit_tiles(a, u);
      tiles[ATTN_FEW] += u.ntiles;
      put_unit(base + s.unit[ATTN_FEW] + size_t(fu) * sizeof(AttnUnit), u);
    }
  }
  if (tid == 0) gstore(toff + s.S, n_units[ATTN_MANY]);
  __syncthreads();

  // units of many rows: the last rows of a sequence, which see most, first
  for (int m = tid; m < n_units[ATTN_MANY]; m += kAttnPlanThreads) {
    int lo = 0, hi = s.S - 1;  // the last sequence whose first unit is not behind m
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (gload<int>(toff + mid) <= m) lo = mid;
      else hi = mid - 1;
    }
    const int first = gload<int>(a.q_off + lo), n = gload<int>(a.q_off + lo + 1) - first;
    const int t = gload<int>(toff + lo + 1) - 1 - m;
    AttnUnit u{first, n, gload<int>(a.lens + lo), t * s.many_rows, 0, lo, 0, 0, 0, 1, 0, {}};
    u.rows = min(s.many_rows, n * s.group - u.row0);
    unit_tiles(a, u);
    tiles[ATTN_MANY] += u.ntiles;
    put_unit(base + s.unit[ATTN_MANY] + size_t(m) * sizeof(AttnUnit), u);
  }
  __syncthreads();

  // pieces
  int n_items[ATTN_KINDS], n_cut[ATTN_KINDS];
#pragma unroll
  for (int kind = 0; kind < ATTN_KINDS; ++kind) {
    int64_t total;
    block_scan(tiles[kind], int64_t(0), part64, [](int64_t x, int64_t y) { return x + y; }, &total);
    const int64_t want = s.target[kind] ? (total + s.target[kind] - 1) / s.target[kind] : 1;
    const int piece = s.cut[kind] ? int(max(want, int64_t(s.least[kind]))) : 0x7fffffff;
    int items = 0, cuts = 0, slots = 0;
    for (int m0 = 0; m0 < n_units[kind]; m0 += kAttnPlanThreads) {
      const int m = m0 + tid;
      char *at = base + s.unit[kind] + size_t(m) * sizeof(AttnUnit);
      int nsplit = 0;
      if (m < n_units[kind]) nsplit = max(1, (gload<int4>(at + 16).z - 1) / piece + 1);
      int all;
      const int item = scan_sum(nsplit, part, &all) + items;
      items += all;
      const int cut = scan_sum(nsplit > 1, part, &all) + cuts;
      cuts += all;
      const int slot = scan_sum(nsplit > 1 ? nsplit : 0, part, &all) + slots;
      slots += all;
      if (nsplit == 0) continue;
      gstore(at + 36, nsplit);
      gstore(at + 40, slot);
      for (int i = 0; i < nsplit; ++i) gstore(base + s.item[kind] + size_t(item + i) * 8, make_int2(m, i));
      if (nsplit > 1) gstore(base + s.cutlist[kind] + size_t(cut) * 4, m);
    }
    n_items[kind] = items;
    n_cut[kind] = cuts;
  }
  int all;
  scan_sum(errors, part, &all);
  if (tid == 0) {
    a.plan[H_ERR] = all;
#pragma unroll
    for (int kind = 0; kind < ATTN_KINDS; ++kind) {
      a.plan[A_ITEMS + kind] = n_items[kind];
      a.plan[A_CUT + kind] = n_cut[kind];
    }
#pragma unroll
    for (int i = 0; i < A_KEYS; ++i) a.plan[A_KEY + i] = a.key[i];
  }
}

}  // namespace

hipError_t launch_attention_plan(const AttnPlanArgs &a, hipStream_t stream) {
  attention_plan_kernel<<<1, kAttnPlanThreads, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace lora
