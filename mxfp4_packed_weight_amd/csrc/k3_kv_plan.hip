// The plan of a decoding step: pages taken and given back, prefix sums,
// slots, positions and tree masks, in one launch.
//
// Everything follows from three prefix sums over the requests (tokens, pages
// taken, pages given back), so no workgroup waits for another: each redoes
// the sums (a thousand requests are 12 KB of reads out of L2 and one scan)
// and then does its own share of the requests' pages or of the tokens. The
// reads and the updates in place do not meet: the ring's taken entries are
// never among those written (count + given back <= n_pages is checked), and
// a table entry is written only past held[r], where no one reads.
//
// The time is that of a launch and of three dependent reads (lengths; table
// or ring; parents): 4.2 us for 16 requests of one token, 8.3 us for 1024
// requests with trees of up to 64 nodes (10.4 where the same workgroups had
// pages and tokens). Masks of more than 64 nodes are kept in memory, a
// dependent read and write for each ancestor: 16 trees of 64 nodes 8.7 us, of
// 65 10.5, of 256 39, of 1024 237; 4 chains of 1024 nodes 731.
#include "k3_kv.h"

namespace k3 {

namespace {

constexpr int kPlanThreads = 1024;  // requests per scan, and tokens per workgroup
constexpr int kPlanWaves = kPlanThreads / 64;
constexpr int kNodes = 32 * K3_MAX_TREE_WORDS;
constexpr uint32_t kCap = 1u << 30;  // sums stop here; x + y <= 2^31 fits

__device__ __forceinline__ uint32_t sat(uint32_t x, uint32_t y) { return min(x + y, kCap); }

// Inclusive sum over a wave's lanes, stopping at kCap (which keeps it
// associative): row shifts, then the rows' last lanes handed on.
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t scan_step(uint32_t v) {
  return sat(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xf, false));
}
__device__ __forceinline__ uint32_t wave_scan(uint32_t v) {
  v = scan_step<0x111, 0xf>(v);
  v = scan_step<0x112, 0xf>(v);
  v = scan_step<0x114, 0xf>(v);
  v = scan_step<0x118, 0xf>(v);
  v = scan_step<0x142, 0xa>(v);  // lane 15 to row 1, lane 47 to row 3
  return scan_step<0x143, 0xc>(v);  // lane 31 to rows 2 and 3
}

__device__ __forceinline__ uint32_t in_ring(uint32_t at, uint32_t N) { return at >= N ? at - N : at; }

struct PlanLds {
  uint32_t cu[kPlanThreads], pops[kPlanThreads], push[kPlanThreads];  // before the request
  int ctx[kPlanThreads], n[kPlanThreads], held[kPlanThreads], need[kPlanThreads];  // need < 0: not served
  uint32_t waves[3][kPlanWaves];
  int missed[kPlanWaves];
  uint32_t taken, given;
  int parents[3 * kNodes];
};
static_assert(kPlanThreads == kNodes, "the parents' window is three spans of tokens");

__global__ __launch_bounds__(kPlanThreads) void kv_plan_kernel(KvPlanArgs a) {
  __shared__ PlanLds L;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int N = a.n_pages, P = a.page;
  int head = a.ring_state[0];
  const int count = min(max(a.ring_state[1], 0), N);
  if (head < 0 || head >= N) head = 0;
  const int token_groups = (a.T + kPlanThreads - 1) / kPlanThreads;
  // the first workgroups take the pages, the others the tokens
  const int page_groups = gridDim.x - token_groups;
  const bool pages = (int)blockIdx.x < page_groups;
  const int t0 = pages ? a.T : (blockIdx.x - page_groups) * kPlanThreads, t = t0 + tid;
  // parents of every node that shares a request with this workgroup's tokens
  if (a.parents && t0 < a.T)
    for (int i = tid; i < 3 * kNodes; i += kPlanThreads) {
      const int s = t0 - kNodes + i;
      L.parents[i] = s >= 0 && s < a.T ? a.parents[s] : -1;
    }
  const int per = (a.R + page_groups - 1) / page_groups;  // requests whose pages are moved here
  const int r_lo = min(a.R, (int)blockIdx.x * per), r_hi = pages ? min(a.R, r_lo + per) : r_lo;
  const bool tells = blockIdx.x == 0;
  if (tid == 0) L.taken = L.given = 0;
  uint32_t cu0 = 0, pops0 = 0, push0 = 0;
  int missed = 0;
  bool placed = false;
  for (int c0 = 0; c0 < a.R; c0 += kPlanThreads) {
    const int r = c0 + tid;
    const bool there = r < a.R;
    const int ctx = there ? a.ctx[r] : 0, raw = there ? a.new_[r] : 0, held = there ? a.held[r] : 0;
    const uint32_t n = min((uint32_t)max(raw, 0), kCap);
    // blocks * P < 2^31, so a length past int is past the table's row
    const uint32_t len = (uint32_t)ctx + (uint32_t)raw;
    const bool sound = ctx >= 0 && raw >= 0 && len <= (uint32_t)(a.blocks * P) && held >= 0 &&
                       held <= a.blocks && !(a.parents && raw > 32 * a.words);
    const int need = sound ? (int)((len + P - 1) / P) : 0;
    const uint32_t pops = sound ? max(need - held, 0) : 0, push = sound ? max(held - need, 0) : 0;
    // the block's exclusive sums
    const uint32_t s0 = wave_scan(n), s1 = wave_scan(min(pops, kCap)), s2 = wave_scan(min(push, kCap));
    __syncthreads();  // the last chunk's readers are done
    if (lane == 63) {
      L.waves[0][wave] = s0;
      L.waves[1][wave] = s1;
      L.waves[2][wave] = s2;
    }
    __syncthreads();
    uint32_t w0 = lane < kPlanWaves ? L.waves[0][lane] : 0, w1 = lane < kPlanWaves ? L.waves[1][lane] : 0,
             w2 = lane < kPlanWaves ? L.waves[2][lane] : 0;
    w0 = wave_scan(w0);
    w1 = wave_scan(w1);
    w2 = wave_scan(w2);
    const uint32_t b0 = wave ? __shfl(w0, wave - 1) : 0, b1 = wave ? __shfl(w1, wave - 1) : 0,
                   b2 = wave ? __shfl(w2, wave - 1) : 0;
    // a sum that stopped says only that it is past every limit: what is
    // before a request is the sum before it, taken from its neighbour
    auto before = [&](uint32_t incl, uint32_t base, uint32_t chunk) {
      uint32_t x = __shfl_up(incl, 1);
      return sat(chunk, sat(base, lane ? x : 0u));
    };
    const uint32_t cu = before(s0, b0, cu0), taken = before(s1, b1, pops0), given = before(s2, b2, push0);
    const bool room = push == 0 || (uint64_t)count + given + push <= (uint64_t)N;
    const bool served = sound && room && (pops == 0 || sat(taken, pops) <= (uint32_t)count);
    L.cu[tid] = there ? cu : 0xffffffffu;
    L.pops[tid] = taken;
    L.push[tid] = given;
    L.ctx[tid] = ctx;
    L.n[tid] = (int)n;
    L.held[tid] = held;
    L.need[tid] = served ? need : -1;
    const uint64_t miss = __ballot(there && !served);
    if (lane == 0) L.missed[wave] = __popcll(miss);
    const uint32_t c_end = sat(cu0, __shfl(w0, kPlanWaves - 1));
    if (tells && there) {
      a.cu[r + 1] = (int)sat(cu, n);
      a.kv_lens[r] = served ? (int)len : 0;
      a.held_out[r] = served ? need : held;
      // served ones come first among those that take (and that give)
      if (served && pops) atomicMax(&L.taken, taken + pops);
      if (served && push) atomicMax(&L.given, given + push);
    }
    __syncthreads();
    if (tells)
      for (int w = 0; w < kPlanWaves; w++) missed += L.missed[w];
    // pages, a wave per request
    for (int rr = max(r_lo, c0) + wave; rr < min(r_hi, c0 + kPlanThreads); rr += kPlanWaves) {
      const int x = rr - c0, nd = L.need[x], hd = L.held[x];
      int32_t *row = a.table + (size_t)rr * a.blocks;
      if (nd < 0) continue;
      // places past the ring's head: below count for pages taken, below N for
      // pages given back, and N <= 2^30, so one subtraction brings them home
      for (int j = lane; j < nd - hd; j += 64) row[hd + j] = a.ring[in_ring(head + L.pops[x] + j, N)];
      for (int j = lane; j < hd - nd; j += 64) a.ring[in_ring(head + count + L.push[x] + j, N)] = row[nd + j];
    }
    // tokens
    if (t < a.T && !placed && (uint32_t)t >= cu0 && (uint32_t)t < c_end) {
      placed = true;
      int lo = 0, hi = min(kPlanThreads, a.R - c0) - 1;  // the last request with cu <= t
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (L.cu[mid] <= (uint32_t)t) lo = mid;
        else hi = mid - 1;
      }
      const int i = t - (int)L.cu[lo];
      const long long p = (long long)L.ctx[lo] + i;
      const int b = (int)p / P;
      int page = -1;  // (not waited for before the tree's walk)
      if (L.need[lo] >= 0)
        page = b < L.held[lo] ? a.table[(size_t)(c0 + lo) * a.blocks + b]
                              : a.ring[in_ring(head + L.pops[lo] + b - L.held[lo], N)];
      int depth = i;
      if (a.parents) {
        const int n_r = L.n[lo], base = tid + kNodes - i;  // node 0 in the window
        int32_t *row = a.mask + (size_t)t * a.words;
        depth = -1;
        int at = i;
        if (n_r > 32 * a.words) {  // not served: no mask
          for (int w = 0; w < a.words; w++) row[w] = 0;
          depth = 0;
        } else if (a.words <= 2) {
          uint64_t bits = 0;
          while (at >= 0 && at < n_r && !((bits >> at) & 1)) {
            bits |= 1ull << at;
            depth++;
            at = L.parents[base + at];
          }
          row[0] = (int32_t)(uint32_t)bits;
          if (a.words == 2) row[1] = (int32_t)(uint32_t)(bits >> 32);
        } else {  // more than 64 nodes: the row itself holds the bits
          for (int w = 0; w < a.words; w++) row[w] = 0;
          while (at >= 0 && at < n_r) {
            const uint32_t word = (uint32_t)row[at >> 5], bit = 1u << (at & 31);
            if (word & bit) break;
            row[at >> 5] = (int32_t)(word | bit);
            depth++;
            at = L.parents[base + at];
          }
        }
      }
      a.slots[t] = page >= 0 && page < N ? page * P + ((int)p - b * P) : -1;
      a.positions[t] = (int)min(max((long long)L.ctx[lo] + depth, -2147483648ll), 2147483647ll);
    }
    cu0 = c_end;
    pops0 = sat(pops0, __shfl(w1, kPlanWaves - 1));
    push0 = sat(push0, __shfl(w2, kPlanWaves - 1));
  }
  if (t < a.T && !placed) {  // past the last request's tokens
    a.slots[t] = -1;
    a.positions[t] = 0;
    if (a.parents)
      for (int w = 0; w < a.words; w++) a.mask[(size_t)t * a.words + w] = 0;
  }
  if (tells && tid == 0) {
    a.cu[0] = 0;
    a.ring_out[0] = (int)in_ring(head + L.taken, N);
    a.ring_out[1] = count - (int)L.taken + (int)L.given;
    a.status[0] = missed;
    a.status[1] = max((int)cu0 - a.T, 0);
  }
}

}  // namespace

hipError_t launch_kv_plan(const KvPlanArgs &a, hipStream_t s) {
  const int grid = (a.T + kPlanThreads - 1) / kPlanThreads + (a.R + kPlanWaves - 1) / kPlanWaves;
  kv_plan_kernel<<<grid, kPlanThreads, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace k3
