// The append to an e4m3 cache with an exponent for each page and head.
//
//   e = ceil(log2(max |x| / 448)) over the page's new rows, not below that of
//   rows that the page has already;  code = e4m3(x 2^-e)
// A wave, or two or four for a larger page, take a page's new rows of one head, keys and
// values: they read them once, keep them in registers while they find the largest
// (pages past that are read again, out of the caches), and write the codes. Only if
// the exponent rises are the page's earlier codes read and rounded again. Which
// page of which request follows without a prefix sum: n tokens touch at most
// n / P + 2 pages, so that request r's are among the numbers from cu[r] / P + 2 r
// on, and a search by 64 finds r.
//
// 20480 tokens of 8 heads of 128 (126 MB): 24 us with warm rows, 5.2 TB/s (a copy:
// 5.1); one token of each of 64 requests 5 us, four dependent reads (lengths,
// table, exponents, codes), and 7 with its call on the host. Few instructions to a
// value made that: sizes are compared two at a time as integers, and rows of
// nothing but ordinary numbers take a way without checks (29 -> 24 us).
#include "k3_kv.h"
#include "k3_lanes.h"
#include "k3_rows.h"

namespace k3 {

namespace {

constexpr int kAppendWaves = 4;
constexpr int kKeep = 4;  // loads of a lane, keys and values alike

// The sizes of 16-bit numbers are in the order of their bits without the sign,
// two to a word. Up to kUsual there is nothing but numbers whose codes are in range.
template <bool BF>
constexpr uint32_t kUsual = BF ? 0x7f7fu : 0x7b80u;  // bf16's largest; 61440
__device__ __forceinline__ uint32_t larger_sizes(uint32_t x, uint32_t y) {
  typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, x), __builtin_bit_cast(u16x2, y)));
}
__device__ __forceinline__ uint32_t largest_bits(const uint4 &x, uint32_t top) {
  constexpr uint32_t kSizes = 0x7fff7fffu;
  return larger_sizes(larger_sizes(larger_sizes(larger_sizes(top, x.x & kSizes), x.y & kSizes), x.z & kSizes), x.w & kSizes);
}
template <bool BF>
__device__ __forceinline__ float of_bits(uint32_t u) {
  if (BF) return __builtin_bit_cast(float, u << 16);
  return (float)__builtin_bit_cast(_Float16, (uint16_t)u);
}
// Eight values' largest size; infinities and NaN do not count.
template <bool BF>
__device__ __forceinline__ float largest(const uint4 &x, float top) {
  float f[8];
  unpack8<BF>(x, f);
#pragma unroll
  for (int j = 0; j < 8; j++) {
    const float y = fabsf(f[j]);
    top = y < INFINITY ? fmaxf(top, y) : top;
  }
  return top;
}
// The byte e + 127 of the smallest 2^e with amax <= 448 2^e = 1.75 2^(e + 8).
__device__ __forceinline__ int exponent_of(float amax) {
  const uint32_t u = __builtin_bit_cast(uint32_t, amax);
  return max((int)(u >> 23) - 8 + ((u & 0x7fffffu) > 0x600000u), 1);
}
template <bool BF>
__device__ __forceinline__ uint2 codes_of(const uint4 &x, int byte, bool usual) {
  float f[8];
  unpack8<BF>(x, f);
  if (usual) {
    const float power = __builtin_bit_cast(float, (uint32_t)(254 - byte) << 23);  // (byte < 254)
#pragma unroll
    for (int j = 0; j < 8; j++) f[j] *= power;
    return to_e4m3(f);
  }
#pragma unroll
  for (int j = 0; j < 8; j++) {
    // (fp16: 448 2^7 < 61440 = 240 2^8 < 65504, which would round to 2^16)
    float y = f[j];
    if (!BF) y = y != y ? y : fminf(fmaxf(y, -61440.f), 61440.f);
    y = ldexpf(y, 127 - byte);
    f[j] = y != y ? y : fminf(fmaxf(y, -448.f), 448.f);
  }
  return to_e4m3(f);
}
// Codes times 2^-fall, rounded again.
__device__ __forceinline__ uint2 lowered(uint2 w, int fall) {
  float f[8];
#pragma unroll
  for (int i = 0; i < 2; i++) {
    const int x = i ? w.y : w.x;
    f[4 * i] = __builtin_amdgcn_cvt_f32_fp8(x, 0);
    f[4 * i + 1] = __builtin_amdgcn_cvt_f32_fp8(x, 1);
    f[4 * i + 2] = __builtin_amdgcn_cvt_f32_fp8(x, 2);
    f[4 * i + 3] = __builtin_amdgcn_cvt_f32_fp8(x, 3);
  }
#pragma unroll
  for (int j = 0; j < 8; j++) f[j] = ldexpf(f[j], -fall);
  return to_e4m3(f);
}

// WAVES: of a page and head; more than one are a workgroup.
template <bool BF, int D, int WAVES>
__global__ __launch_bounds__(64 * kAppendWaves) void kv_append_kernel(KvAppendArgs a, int items) {
  constexpr int LPR = D / 8, RPL = 64 / LPR;  // lanes of a row, rows of a load
  const int lane = threadIdx.x & 63, sub = lane / LPR, d0 = lane % LPR * 8;
  const int H = a.c.n_heads, P = a.c.page_size;
  // (below 2^29 in all: T / 4 and 2 R items, 2^10 heads)
  const int wave = threadIdx.x >> 6, part = WAVES == 1 ? 0 : wave;
  const int group = blockIdx.y * gridDim.x + blockIdx.x;
  const int unit = __builtin_amdgcn_readfirstlane(WAVES == 1 ? group * kAppendWaves + wave : group);
  const int item = unit / H, h = unit - item * H;
  if (item >= items) return;
  auto start = [&](int r) { return min(max(a.cu[r], 0), a.T) / P + 2 * r; };
  // the last request that starts at or before the item
  int r = 0;
  for (int n = a.R; n > 1;) {
    const int step = (n + 63) / 64;
    const uint64_t at = __ballot(lane * step < n && start(min(r + lane * step, a.R - 1)) <= item);
    if (!at) return;
    const int last = 63 - __builtin_clzll(at);
    r += last * step;
    n = min(step, n - last * step);
  }
  const int t0 = a.cu[r], len = a.kv_lens[r];
  const int64_t n = (int64_t)a.cu[r + 1] - t0;
  if (t0 < 0 || n <= 0 || t0 + n > a.T || len < n || len > a.blocks * P) return;
  const int ctx = len - (int)n, j = item - (t0 / P + 2 * r), b = ctx / P + j;
  if (j < 0 || b > (len - 1) / P) return;
  const int page = a.table[(int64_t)r * a.blocks + b];
  const int first = max(ctx, b * P), rows = min(len, b * P + P) - first, earlier = first - b * P;
  const int t = t0 + first - ctx;
  const uint16_t *in[2] = {a.k + t * a.k_stride + h * D + d0, a.v + t * a.v_stride + h * D + d0};
  const int64_t in_stride[2] = {a.k_stride, a.v_stride};
  uint4 x[2][kKeep];
  auto load = [&](int i0) {
#pragma unroll
    for (int i = 0; i < kKeep; i++)
#pragma unroll
      for (int s = 0; s < 2; s++) {
        const int row = i0 + (part * kKeep + i) * RPL + sub;
        x[s][i] = uint4{0, 0, 0, 0};
        if (row < rows) x[s][i] = *(const uint4 *)(in[s] + row * in_stride[s]);
      }
  };
  load(0);  // (on their way while the page is looked up)
  if (page < 0 || page >= a.c.n_pages) return;
  const int64_t at = page * a.c.page_stride + h * a.c.head_stride + d0;
  uint8_t *out[2] = {(uint8_t *)a.c.k + at, (uint8_t *)a.c.v + at};
  uint8_t *exps[2] = {a.k_exp + (int64_t)page * H + h, a.v_exp + (int64_t)page * H + h};

  int was[2] = {0, 0};  // the earlier rows' exponents
  if (earlier)
#pragma unroll
    for (int s = 0; s < 2; s++) was[s] = min(max((int)*exps[s], 1), 254);
  constexpr int CHUNK = WAVES * kKeep * RPL;
  uint32_t bits[2] = {0, 0};
  for (int i0 = 0; i0 < rows; i0 += CHUNK) {
    if (i0) load(i0);
#pragma unroll
    for (int i = 0; i < kKeep; i++)
#pragma unroll
      for (int s = 0; s < 2; s++) bits[s] = largest_bits(x[s][i], bits[s]);
  }
  // the waves' largest: of bits, and of numbers where there are others among them
  auto of_all = [&](uint32_t (&v)[2]) {
#pragma unroll
    for (int s = 0; s < 2; s++)
      halving<32>([&](auto d) { v[s] = max(v[s], lane_xor<decltype(d)::value>(v[s])); });
    if constexpr (WAVES > 1) {  // (they all come here: they have one page)
      __shared__ uint32_t tops[WAVES][2];
      __syncthreads();
      if (lane < 2) tops[wave][lane] = lane ? v[1] : v[0];
      __syncthreads();
      for (int i = 0; i < WAVES; i++)
#pragma unroll
        for (int s = 0; s < 2; s++) v[s] = max(v[s], tops[i][s]);
    }
  };
#pragma unroll
  for (int s = 0; s < 2; s++) bits[s] = max(bits[s] & 0xffffu, bits[s] >> 16);
  of_all(bits);
  float top[2] = {of_bits<BF>(bits[0]), of_bits<BF>(bits[1])};
  bool usual = max(bits[0], bits[1]) <= kUsual<BF>;
  if (!usual) {
    float most[2] = {0.f, 0.f};
    for (int i0 = 0; i0 < rows; i0 += CHUNK) {
      if (rows > CHUNK) load(i0);
#pragma unroll
      for (int i = 0; i < kKeep; i++)
#pragma unroll
        for (int s = 0; s < 2; s++) most[s] = largest<BF>(x[s][i], most[s]);
    }
    // (numbers that are not negative are in the order of their bits)
    uint32_t u[2] = {__builtin_bit_cast(uint32_t, most[0]), __builtin_bit_cast(uint32_t, most[1])};
    of_all(u);
    top[0] = __builtin_bit_cast(float, u[0]);
    top[1] = __builtin_bit_cast(float, u[1]);
  }
  int byte[2];
#pragma unroll
  for (int s = 0; s < 2; s++) {
    byte[s] = max(exponent_of(top[s]), was[s]);
    usual &= byte[s] < 254;
    if (lane == 0 && part == 0) *exps[s] = (uint8_t)byte[s];
    if (earlier && byte[s] > was[s])
      for (int row = part * RPL + sub; row < earlier; row += WAVES * RPL) {
        uint2 *p = (uint2 *)(out[s] + row * a.c.slot_stride);
        *p = lowered(*p, byte[s] - was[s]);
      }
  }
  for (int i0 = 0; i0 < rows; i0 += CHUNK) {
    if (rows > CHUNK) load(i0);
#pragma unroll
    for (int i = 0; i < kKeep; i++)
#pragma unroll
      for (int s = 0; s < 2; s++) {
        const int row = i0 + (part * kKeep + i) * RPL + sub;
        if (row < rows) *(uint2 *)(out[s] + (earlier + row) * a.c.slot_stride) = codes_of<BF>(x[s][i], byte[s], usual);
      }
  }
}

template <bool BF, int D>
void launch(const KvAppendArgs &a, int items, hipStream_t s) {
  const unsigned units = (unsigned)items * a.c.n_heads;
  // A wave keeps kKeep loads of 512 / D rows. 20480 tokens of 8 heads of 128, pages
  // of 16 / 32 / 64 places: 24 / 22 / 22 us (before the last step 30 / 28 / 28, and with
  // one wave and eight loads 39 / 33 / 35).
  const int most = kKeep * 512 / D, P = a.c.page_size;
  // (2^32 threads do not fit into one dimension of a launch: 2^18 pages of 256 heads have them)
  auto grid = [](unsigned groups) {
    constexpr unsigned kRow = 1u << 23;
    return dim3(groups < kRow ? groups : kRow, (groups + kRow - 1) / kRow);
  };
  if (P <= most)
    kv_append_kernel<BF, D, 1><<<grid((units + kAppendWaves - 1) / kAppendWaves), 64 * kAppendWaves, 0, s>>>(a, items);
  else if (P <= 2 * most) kv_append_kernel<BF, D, 2><<<grid(units), 128, 0, s>>>(a, items);
  else kv_append_kernel<BF, D, 4><<<grid(units), 256, 0, s>>>(a, items);
}

template <bool BF>
hipError_t by_dim(const KvAppendArgs &a, hipStream_t s) {
  const int items = a.T / a.c.page_size + 2 * a.R;
  switch (a.c.head_dim) {
    case 64: launch<BF, 64>(a, items, s); break;
    case 128: launch<BF, 128>(a, items, s); break;
    default: launch<BF, 256>(a, items, s);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_kv_append(const KvAppendArgs &a, hipStream_t s) {
  return a.dtype == K3_BF16 ? by_dim<true>(a, s) : by_dim<false>(a, s);
}

}  // namespace k3
