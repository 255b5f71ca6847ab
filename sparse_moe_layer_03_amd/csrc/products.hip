// Products C = A B^T on the matrix cores, dense or grouped by expert over ragged row counts, in bf16 with fp32
// sums or in 8-bit integers with int32 sums and a scale per A row and per B row.
//
// Both types move the same bytes: a lane feeds 16 bytes of a row (8 bf16 or 16 codes) to one 32 x 32 matrix
// instruction, so tiles, staging and addressing below count bytes and only the instruction and the epilogue
// differ.  B (the weights) is the instruction's first operand: a lane then holds, of one output row, four
// consecutive columns per register group.
//
// Grouped: expert e owns positions off[e] .. off[e] + count(e) - 1.  Position p is output row id = rows[p] (or p)
// and reads A row id / a_div; ids outside [0, R) are padding and are skipped.
#include <atomic>

#include "block_internal.h"
#include "product_rule.h"

namespace moe {
namespace {

typedef int i32x16 __attribute__((ext_vector_type(16)));
typedef int i32x4v __attribute__((ext_vector_type(4)));

template <bool I8>
struct Acc {
  typedef f32x16 t32;
};
template <>
struct Acc<true> {
  typedef i32x16 t32;
};

__device__ __forceinline__ f32x16 mma32(const u32x4& b, const u32x4& a, const f32x16& c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, b), __builtin_bit_cast(bf16x8, a), c, 0, 0,
                                                 0);
}
__device__ __forceinline__ i32x16 mma32(const u32x4& b, const u32x4& a, const i32x16& c) {
  return __builtin_amdgcn_mfma_i32_32x32x32_i8(__builtin_bit_cast(i32x4v, b), __builtin_bit_cast(i32x4v, a), c, 0, 0,
                                               0);
}

__device__ const u32x4 kZeros[1] = {{0u, 0u, 0u, 0u}};  // source of the chunks behind a row's end

// The positions of a run that begins at off, cut to [0, P): n of them, or up to n where it is the run's end.  No step
// leaves an int, whatever the three values hold.
__device__ __forceinline__ void cut_run(int P, int off, int n, bool is_end, int& first, int& count) {
  first = min(max(off, 0), P);
  const int len = is_end ? max(n, first) - first : max(n, 0) + min(off, 0);
  count = min(max(len, 0), P - first);
}

// Positions of expert e.
__device__ __forceinline__ void expert_range(const ProductArgs& p, int e, int& first, int& count) {
  cut_run(p.P, p.off[e], p.counts ? p.counts[e] : p.off[e + 1], !p.counts, first, count);
}

// The same for an expert that is the same in all lanes, by scalar loads: a vector load would wait behind the ring's.
// (First positions and counts kept in registers like the starts cost as much time and spill in the largest tile.)
__device__ __forceinline__ void expert_range_scalar(const ProductArgs& p, int e, int& first, int& count) {
  typedef const __attribute__((address_space(4))) int32_t* scalar_ptr;
  const scalar_ptr off = (scalar_ptr)(uintptr_t)p.off, counts = (scalar_ptr)(uintptr_t)p.counts;
  cut_run(p.P, off[e], p.counts ? counts[e] : off[e + 1], !p.counts, first, count);
}

// Output row of a position, -1 for padding.
__device__ __forceinline__ int output_row(const ProductArgs& p, int pos) {
  const int id = p.rows ? p.rows[pos] : pos;
  return (unsigned)id < (unsigned)p.R ? id : -1;
}

// A row of an output row: id / a_div by a multiplication (exact for id < 2^31; div_mul 0: a_div is 1).
__device__ __forceinline__ int a_row(const ProductArgs& p, int id) {
  return p.div_mul ? (int)(__umulhi((unsigned)id, p.div_mul) >> p.div_shift) : id;
}

// One 32 x 32 block of outputs: lane l holds, of row l & 31, columns n + 8 g + 4 (l >> 5) + i in register 4 g + i.
// To memory a lane moves 16 bytes of bf16 twice: columns n + 8 (l >> 5) + (l & 16) .. + 7 of rows l & 15 and
// 16 + (l & 15), so that 4 lanes cover 64 contiguous bytes of a row.  The lane halves exchange register groups and
// lanes 16 apart exchange the resulting chunks; both exchanges undo themselves.
struct BlockRows {
  int id, id_lo, id_hi;  // output rows of block rows l & 31, l & 15 and 16 + (l & 15); < 0: none
};
// lanes 0-31 of words i + 2 with lanes 32-63 of words i
__device__ __forceinline__ void swap_halves(u32x4& v) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const auto x = __builtin_amdgcn_permlane32_swap(v[i], v[i + 2], false, false);
    v[i] = x[0], v[i + 2] = x[1];
  }
}
// lanes 0-15 and 32-47 of b with lanes 16-31 and 48-63 of a
__device__ __forceinline__ void swap_rows(u32x4& a, u32x4& b) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const auto x = __builtin_amdgcn_permlane16_swap(a[i], b[i], false, false);
    a[i] = x[0], b[i] = x[1];
  }
}

// The addend of a block as it lies in memory.
struct BlockAdd {
  u32x4 lo, hi;
};
__device__ __forceinline__ BlockAdd load_add(const ProductArgs& p, const BlockRows& r, int n, int lane) {
  const int col = n + 8 * (lane >> 5) + (lane & 16);
  BlockAdd a = {{0u, 0u, 0u, 0u}, {0u, 0u, 0u, 0u}};
  if (p.add && r.id_lo >= 0 && col < p.N) a.lo = *reinterpret_cast<const u32x4*>(p.add + (size_t)r.id_lo * p.N + col);
  if (p.add && r.id_hi >= 0 && col < p.N) a.hi = *reinterpret_cast<const u32x4*>(p.add + (size_t)r.id_hi * p.N + col);
  return a;
}

// sa: the row's scale; sb, sbias: the block's 32 column scales and biases in LDS.  All lanes take part.
template <bool I8, bool F32, bool EPI, class A>
__device__ __forceinline__ void store_block(const ProductArgs& p, const BlockRows& r, float sa, const float* sb,
                                            const float* sbias, BlockAdd ad, int n, int lane, const A& acc) {
  const int h = lane >> 5;
  float v[4][4];
  if constexpr (EPI) {
    swap_rows(ad.lo, ad.hi);
    swap_halves(ad.lo), swap_halves(ad.hi);
  }
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    if constexpr (I8) {
      const float4 f4 = *reinterpret_cast<const float4*>(sb + 8 * g + 4 * h);
      const float f[4] = {f4.x, f4.y, f4.z, f4.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) v[g][i] = (float)acc[4 * g + i] * sa * f[i];
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[g][i] = acc[4 * g + i];
    }
    if constexpr (EPI) {
      // register group g of the addend: words 0, 1 (even g) or 2, 3 (odd g) of its half
      const u32x4& w = g < 2 ? ad.lo : ad.hi;
      const uint32_t w0 = w[2 * (g & 1)], w1 = w[2 * (g & 1) + 1];
      const float4 b = *reinterpret_cast<const float4*>(sbias + 8 * g + 4 * h);
      v[g][0] = v[g][0] + b.x + bf16_to_f32((uint16_t)w0), v[g][1] = v[g][1] + b.y + bf16_to_f32((uint16_t)(w0 >> 16));
      v[g][2] = v[g][2] + b.z + bf16_to_f32((uint16_t)w1), v[g][3] = v[g][3] + b.w + bf16_to_f32((uint16_t)(w1 >> 16));
    }
    if constexpr (F32) {
      const int col = n + 8 * g + 4 * h;
      if (r.id >= 0 && col < p.N)
        *reinterpret_cast<float4*>(static_cast<float*>(p.c) + (size_t)r.id * p.N + col) =
            make_float4(v[g][0], v[g][1], v[g][2], v[g][3]);
    }
  }
  if constexpr (!F32) {
    u32x4 lo, hi;
    lo[0] = cvt_bf16x2(v[0][0], v[0][1]), lo[1] = cvt_bf16x2(v[0][2], v[0][3]);
    lo[2] = cvt_bf16x2(v[1][0], v[1][1]), lo[3] = cvt_bf16x2(v[1][2], v[1][3]);
    hi[0] = cvt_bf16x2(v[2][0], v[2][1]), hi[1] = cvt_bf16x2(v[2][2], v[2][3]);
    hi[2] = cvt_bf16x2(v[3][0], v[3][1]), hi[3] = cvt_bf16x2(v[3][2], v[3][3]);
    swap_halves(lo), swap_halves(hi);
    swap_rows(lo, hi);
    const int col = n + 8 * h + (lane & 16);
    uint16_t* c = static_cast<uint16_t*>(p.c);
    if (r.id_lo >= 0 && col < p.N) *reinterpret_cast<u32x4*>(c + (size_t)r.id_lo * p.N + col) = lo;
    if (r.id_hi >= 0 && col < p.N) *reinterpret_cast<u32x4*>(c + (size_t)r.id_hi * p.N + col) = hi;
  }
}

// ---------------------------------------------------------------------------------------------------------------
// Few rows (dense 8-bit products): a workgroup owns 16 columns and reads their weights once, straight into
// registers.  Its four waves take every fourth 128-byte line of the rows (two 16 x 16 matrix instructions deep), U
// lines at a time, and add their partial sums through LDS.  One row by 2048 x 4096 takes 3.2 us, a launch and one round
// of loads; the bytes alone would take 1.8.

typedef int i32x4 __attribute__((ext_vector_type(4)));

template <bool F32, bool EPI, int MT, int U>
__global__ __launch_bounds__(256) void skinny_kernel(ProductArgs p) {
  constexpr int W = 4;
  __shared__ i32x4 part[W][MT][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int n0 = blockIdx.x * 16, k0 = (lane >> 4) * 16;
  const char* zeros = reinterpret_cast<const char*>(kZeros);
  const char* b = static_cast<const char*>(p.b) + (size_t)min(n0 + (lane & 15), p.N - 1) * p.Kb;
  const char* a[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
    a[m] = static_cast<const char*>(p.a) + (size_t)min(16 * m + (lane & 15), p.P - 1) * p.Kb;
  const int lines = (p.Kb + 127) / 128;
  i32x4 acc[MT] = {};
  for (int l0 = wave; l0 < lines; l0 += W * U) {
    u32x4 fb[U][2], fa[MT][U][2];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int k = (l0 + u * W) * 128 + h * 64 + k0;
        const bool in = k < p.Kb;
        fb[u][h] = *reinterpret_cast<const u32x4*>(in ? b + k : zeros);
#pragma unroll
        for (int m = 0; m < MT; ++m) fa[m][u][h] = *reinterpret_cast<const u32x4*>(in ? a[m] + k : zeros);
      }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int m = 0; m < MT; ++m)
          acc[m] = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, fb[u][h]),
                                                         __builtin_bit_cast(i32x4, fa[m][u][h]), acc[m], 0, 0, 0);
  }
#pragma unroll
  for (int m = 0; m < MT; ++m) part[wave][m][lane] = acc[m];
  __syncthreads();
  // wave m adds and stores row block m: lane l holds, of row l & 15, columns 4 (l >> 4) + i
  for (int m = wave; m < MT; m += W) {
    const i32x4 s = (part[0][m][lane] + part[1][m][lane]) + (part[2][m][lane] + part[3][m][lane]);
    const int id = 16 * m + (lane & 15), n = n0 + 4 * (lane >> 4);
    if (id >= p.P || n >= p.N) continue;
    const size_t at = (size_t)id * p.N + n;
    const float sa = p.a_scale[id];
    const float4 f = *reinterpret_cast<const float4*>(p.b_scale + n);
    float v[4] = {(float)s[0] * sa * f.x, (float)s[1] * sa * f.y, (float)s[2] * sa * f.z, (float)s[3] * sa * f.w};
    if constexpr (EPI) {
      if (p.bias) {
        const float4 t = *reinterpret_cast<const float4*>(p.bias + n);
        v[0] += t.x, v[1] += t.y, v[2] += t.z, v[3] += t.w;
      }
      if (p.add) {
        const u32x2 w = *reinterpret_cast<const u32x2*>(p.add + at);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] += bf16_to_f32((uint16_t)(w[i >> 1] >> (16 * (i & 1))));
      }
    }
    if constexpr (F32)
      *reinterpret_cast<float4*>(static_cast<float*>(p.c) + at) = make_float4(v[0], v[1], v[2], v[3]);
    else
      *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(p.c) + at) =
          u32x2{cvt_bf16x2(v[0], v[1]), cvt_bf16x2(v[2], v[3])};
  }
}

// ---------------------------------------------------------------------------------------------------------------
// Persistent kernel: BM x BN tiles, operands loaded straight into an S-stage ring in LDS, loads S - 1 steps ahead also
// across items, one barrier per K step.
//
// What bounds it: dense 8-bit 8192 x 4096 x 4096 takes 122 us (2.25 POP/s; a library's product 131 us); with the matrix
// instructions taken out of a copy 98 us, with the loads taken out 95 us, with loads and LDS reads out 74 us: the parts
// overlap to within a quarter.  Grouped bf16 gate/up rows of 8192 tokens (256 experts, top-8, most of them small) take
// 367 us, 345 without the matrix instructions: 1.44 GB are read past the L2 caches and 0.135 written, 4.3 TB/s where a
// plain read of 4 GiB reaches 6.8 (a direct-to-LDS load from L2 alone 127 GB/s per CU); the two-stage ring waits for
// all loads at every step, and half of the experts fill a tile to less than a sixth.  Below a mean of about 64 rows per
// expert the weights' stream is all: 32 tokens, some 77 experts, 55 us, 5.9 TB/s (a plain read of as much 5.9).
//
// Measured and not taken, dense / grouped in us against 128 / 390: four waves of 128 x 128 (spills) 143 / 457; loads
// spread between the matrix instructions 134 / 425; the last sub-step's instructions behind the barrier 131 / 404;
// items dealt cyclically over the XCDs (even, but fewer L2 hits) - / 407; small tiles on a deeper ring of their own - /
// 414; skipping the loads of padding rows 133 / 410.  Leaving an item's stores in flight over the next item's first
// steps: 123 / 374 against 122 / 372 by then (3% less with an addend, nothing elsewhere).

// 16 (4) bytes per lane from src to LDS at lds_base + 16 (4) * lane; lds_base is wave-uniform.  Inline assembly, so
// that the compiler's wait counts do not order LDS reads behind loads in flight; the K loop waits itself.
__device__ __forceinline__ void to_lds16(const void* src, uint32_t lds_base) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(lds_base), "v"(src)
               : "memory", "m0");
}
__device__ __forceinline__ void to_lds4(const void* src, uint32_t lds_base) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off" ::"s"(lds_base), "v"(src)
               : "memory", "m0");
}
// The K loop's form: a wave-uniform base and 32-bit lane offsets that stay the same from step to step, so that a load
// costs no vector instruction (dense 8-bit 8192 x 4096 x 4096 132 -> 124 us, grouped bf16 prefill 394 -> 376 us).
// NT: past the caches.
template <bool NT>
__device__ __forceinline__ void to_lds16(const char* base, uint32_t off, uint32_t lds_base) {
  if constexpr (NT)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2 nt" ::"s"(lds_base), "v"(off), "s"(base)
                 : "memory", "m0");
  else
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(lds_base), "v"(off), "s"(base)
                 : "memory", "m0");
}
template <int N>
__device__ __forceinline__ void wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// A K step is 128 bytes of a row, 8 chunks of 16.  (64-byte steps in twice the stages read every cache line in two
// halves: dense 8-bit 8192 x 4096 x 4096 145 -> 157 us.)
constexpr int kCh = 8;
// In LDS chunk c of a row lies at c ^ swz_term(row): any 16 consecutive rows read at one chunk hit 16 distinct bank
// groups.
__device__ __forceinline__ int swz_term(int row) { return ((row >> 1) ^ ((row & 1) << 2)) & 7; }

// Row tiles of an expert whose items run together over all column blocks, so that the 32 workgroups of an XCD read
// few distinct rows and columns at a time.
constexpr int kGroupM = 4;

struct ProductItem {
  int expert, first, rows, n0;
  int only;  // the expert's only tile
};

// The item list of a launch: experts in order, within an expert groups of kGroupM row tiles, within a group column
// blocks, within a block the group's tiles.  Lane l of every wave keeps the starts of experts 4 l .. 4 l + 3
// in registers; each is read from its lane before one is selected, since a selection among the array's elements
// would put it into scratch memory, whose loads wait behind the ring's (down rows of a chunk 48.0 -> 43.6 us).  One form
// uses scratch memory still: fp32 output with bias or addend on the largest tile spills 4 or 6 registers around its
// epilogue (8192 x 4096 x 4096 with addend 181 us against 150 to bf16, without 136 against 122).
template <int BM, int BN>
struct ProductList {
  int nbn, total;
  int start[4];  // index of the expert's first item

  __device__ __forceinline__ void init(const ProductArgs& p, int lane) {
    nbn = (p.N + BN - 1) / BN;
    if (!p.off) {
      total = ((p.P + BM - 1) / BM) * nbn;
      return;
    }
    int sum = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = 4 * lane + i;
      int first = 0, count = 0;
      if (e < p.E) expert_range(p, e, first, count);
      start[i] = sum;
      // the launch keeps experts that share the positions below the bound; it keeps 256 counts in an int whatever
      // off and counts hold
      const int64_t items = (int64_t)((count + BM - 1) / BM) * nbn;
      sum += (int)(items < kMaxItems ? items : kMaxItems - 1);
    }
    int incl = sum;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_up(incl, d);
      if (lane >= d) incl += o;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) start[i] += incl - sum;
    total = __builtin_amdgcn_readlane(incl, 63);
  }

  __device__ __forceinline__ ProductItem at(const ProductArgs& p, int item) const {
    ProductItem it;
    int j = item, rows = p.P, base = 0;
    it.expert = 0;
    if (p.off) {
      // of the experts that start at or before the item the last one holds it: an empty one starts where the next does
      int n = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) n += __popcll(__ballot(start[i] <= item));
      it.expert = min(n, p.E) - 1;
      const int l = it.expert >> 2, q = it.expert & 3;
      const int s0 = __builtin_amdgcn_readlane(start[0], l), s1 = __builtin_amdgcn_readlane(start[1], l);
      const int s2 = __builtin_amdgcn_readlane(start[2], l), s3 = __builtin_amdgcn_readlane(start[3], l);
      j -= q < 2 ? (q == 0 ? s0 : s1) : (q == 2 ? s2 : s3);
      expert_range_scalar(p, it.expert, base, rows);
    }
    const int tiles = (rows + BM - 1) / BM;
    const int g = j / (kGroupM * nbn);
    const int size = min(kGroupM, tiles - g * kGroupM);
    const int rem = j - g * kGroupM * nbn;
    const int m = g * kGroupM + rem % size;
    it.n0 = (rem / size) * BN;
    it.first = base + m * BM;
    it.rows = min(BM, rows - m * BM);
    it.only = tiles == 1;
    return it;
  }
};

template <bool I8, bool EPI, int BM, int BN, int WM, int WN, int S>
struct RingCfg {
  static constexpr int NW = WM * WN, NT = NW * 64, MI = BM / WM / 32, NJ = BN / WN / 32;
  static constexpr int RPI = 64 / kCh;  // rows one load instruction fills
  static constexpr int NA = BM / RPI / NW, NB = BN / RPI / NW;  // load instructions per wave and step
  static constexpr int STAGE = (BM + BN) * kCh;  // chunks
  static constexpr int SUB = kCh / 2;  // matrix instructions deep per step
  // LDS: stages, output rows of three items, scales and biases of two items
  static constexpr size_t LDS =
      (size_t)S * STAGE * 16 + 3 * BM * 4 + (I8 ? 2 * (BM + BN) * 4 : 0) + (EPI ? 2 * BN * 4 : 0);
  static constexpr int PER_CU = LDS * 2 <= 160 * 1024 ? 2 : 1;
  static_assert(BM % (RPI * NW) == 0 && BN % (RPI * NW) == 0 && BN <= NT && BM <= NT && LDS <= 160 * 1024, "");
};

template <bool I8, bool F32, bool EPI, bool NT, bool TAIL, int BM, int BN, int WM, int WN, int S>
__global__ __launch_bounds__(WM* WN * 64, 1) void ring_kernel(ProductArgs p) {
  using C = RingCfg<I8, EPI, BM, BN, WM, WN, S>;
  extern __shared__ __align__(16) unsigned char smem[];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / WN, wn = wave % WN;

  ProductList<BM, BN> list;
  list.init(p, lane);
  // each XCD takes one contiguous run of items, its workgroups every nslot-th of them
  const int per = (list.total + kNumXcd - 1) / kNumXcd;
  const int nslot = (int)gridDim.x / kNumXcd;
  const int xcd = (int)blockIdx.x % kNumXcd;
  const int begin = xcd * per + (int)blockIdx.x / kNumXcd;
  const int end = min(list.total, (xcd + 1) * per);
  if (begin >= end) return;
  const int n_items = (end - begin + nslot - 1) / nslot;

  u32x4* sm = reinterpret_cast<u32x4*>(smem);
  int* s_ids = reinterpret_cast<int*>(smem + (size_t)S * C::STAGE * 16);  // [3][BM]
  float* s_sa = reinterpret_cast<float*>(s_ids + 3 * BM);                // [2][BM]
  float* s_sb = s_sa + 2 * BM;                                           // [2][BN]
  float* s_bias = s_sb + 2 * BN;                                         // [2][BN]
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) unsigned char*)smem;
  const uint32_t lds_ids = lds0 + S * C::STAGE * 16, lds_sa = lds_ids + 3 * BM * 4;
  const uint32_t lds_sb = lds_sa + 2 * BM * 4, lds_bias = lds_sb + 2 * BN * 4;

  // at least S - 1 steps per item (those behind the row's end read zeros), so that an item's row ids have landed
  // when its loads begin and no buffer of an item is refilled before its epilogue
  const int nk = max((p.Kb + kCh * 16 - 1) / (kCh * 16), S - 1);
  // TAIL: steps without a row's end in them, and whether every A offset fits 32 bits
  const int full = p.Kb / (kCh * 16);
  const bool narrow = !TAIL || ((uint64_t)a_row(p, p.R - 1) + 1) * p.Kb <= (1ull << 32);

  // ---- loads
  ProductItem lit = {};  // the item being loaded
  ProductItem nit = list.at(p, begin);  // the one after it
  int l_index = -1, l_kb = nk;
  // byte offsets of this lane's rows from A and from the item's first B row
  typedef std::conditional_t<TAIL, uint64_t, uint32_t> aoff_t;
  aoff_t aoff[C::NA];
  uint32_t boff[C::NB];
  const char* abase = static_cast<const char*>(p.a);
  const char* bbase = abase;
  const int lrow = lane / kCh;  // row of this lane within a load instruction
  auto chunk = [&](int r) { return (lane % kCh) ^ swz_term(r); };  // logical chunk this lane fetches of row r
  // this lane's 16 bytes at off, or zeros where they lie behind the row's end; r: the load's first tile row
  auto source = [&](const char* base, uint64_t off, int r) {
    const int k = l_kb * (kCh * 16);
    return k + chunk(r + lrow) * 16 < p.Kb ? base + off + k : reinterpret_cast<const char*>(kZeros);
  };
  auto load_ids = [&](int index, const ProductItem& it) {
    const int r = wave * 64 + lane;
    if (p.rows && r < BM)
      to_lds4(p.rows + it.first + min(r, it.rows - 1), lds_ids + (uint32_t)((index % 3) * BM + wave * 64) * 4);
  };
  auto row_id = [&](int index, const ProductItem& it, int r) {  // output row of tile row r, -1: none
    const int id = p.rows ? s_ids[(index % 3) * BM + r] : it.first + r;
    return r < it.rows && (unsigned)id < (unsigned)p.R ? id : -1;
  };
  // starts the next item: sources of its rows; its scales and the row ids of the one after it into LDS
  auto next_item = [&]() {
    ++l_index;
    l_kb = 0;
    lit = nit;
    if (l_index + 1 < n_items) {
      nit = list.at(p, begin + (l_index + 1) * nslot);
      load_ids(l_index + 1, nit);
    }
#pragma unroll
    for (int q = 0; q < C::NA; ++q) {
      const int r = (wave * C::NA + q) * C::RPI + lrow;
      const int id = max(row_id(l_index, lit, r), 0);  // rows without data read row 0
      aoff[q] = (aoff_t)((uint64_t)a_row(p, id) * p.Kb + chunk(r) * 16);
    }
    bbase = static_cast<const char*>(p.b) + ((size_t)lit.expert * p.N + lit.n0) * p.Kb;
#pragma unroll
    for (int q = 0; q < C::NB; ++q) {
      const int r = (wave * C::NB + q) * C::RPI + lrow;
      boff[q] = (uint32_t)(min(r, p.N - 1 - lit.n0) * p.Kb + chunk(r) * 16);
    }
    if constexpr (I8) {
      const int par = l_index & 1, r = wave * 64 + lane;
      if (r < BM)
        to_lds4(p.a_scale + a_row(p, max(row_id(l_index, lit, r), 0)), lds_sa + (uint32_t)(par * BM + wave * 64) * 4);
      if (r < BN)
        to_lds4(p.b_scale + (size_t)lit.expert * p.N + min(lit.n0 + r, p.N - 1),
                lds_sb + (uint32_t)(par * BN + wave * 64) * 4);
      if (EPI && r < BN)
        to_lds4(p.bias ? static_cast<const void*>(p.bias + min(lit.n0 + r, p.N - 1)) : kZeros,
                lds_bias + (uint32_t)(par * BN + wave * 64) * 4);
    }
  };
  // The loads of one operand of a step.  Behind the last item they repeat its last step (TAIL: read zeros).
  auto issue_a = [&](int slot) {
    const uint32_t dst = lds0 + (uint32_t)slot * (C::STAGE * 16) + (uint32_t)(wave * C::NA * C::RPI * kCh) * 16;
    const char* base = abase + min(l_kb, nk - 1) * (kCh * 16);
    if (TAIL && (l_kb >= full || !narrow)) {
#pragma unroll
      for (int q = 0; q < C::NA; ++q)
        to_lds16(source(abase, aoff[q], (wave * C::NA + q) * C::RPI), dst + (uint32_t)(q * C::RPI * kCh) * 16);
    } else {
#pragma unroll
      for (int q = 0; q < C::NA; ++q)
        to_lds16<false>(base, (uint32_t)aoff[q], dst + (uint32_t)(q * C::RPI * kCh) * 16);
    }
  };
  auto issue_b = [&](int slot) {
    const uint32_t dst = lds0 + (uint32_t)slot * (C::STAGE * 16) + (uint32_t)((BM + wave * C::NB * C::RPI) * kCh) * 16;
    const char* base = bbase + min(l_kb, nk - 1) * (kCh * 16);
    if (TAIL && l_kb >= full) {
#pragma unroll
      for (int q = 0; q < C::NB; ++q)
        to_lds16(source(bbase, boff[q], (wave * C::NB + q) * C::RPI), dst + (uint32_t)(q * C::RPI * kCh) * 16);
    } else if (NT && lit.only) {
#pragma unroll
      for (int q = 0; q < C::NB; ++q) to_lds16<true>(base, boff[q], dst + (uint32_t)(q * C::RPI * kCh) * 16);
    } else {
#pragma unroll
      for (int q = 0; q < C::NB; ++q) to_lds16<false>(base, boff[q], dst + (uint32_t)(q * C::RPI * kCh) * 16);
    }
    ++l_kb;
  };

  // ---- fragments: tile row block b holds rows 32 b ..; blocks are dealt to the waves in turn, so that a partly
  // filled tile gives every wave its share of the filled blocks
  const int frow = lane & 31;
  struct Frag {
    u32x4 a[C::MI], b[C::NJ];
  };
  auto read_frags = [&](Frag& f, const u32x4* st, int sub) {
    const int c = frow * kCh + ((2 * sub + (lane >> 5)) ^ swz_term(frow));
#pragma unroll
    for (int m = 0; m < C::MI; ++m) f.a[m] = st[(m * WM + wm) * 32 * kCh + c];
#pragma unroll
    for (int j = 0; j < C::NJ; ++j) f.b[j] = st[(BM + (wn * C::NJ + j) * 32) * kCh + c];
  };

  // ---- start: the first item's row ids, then S - 1 steps of loads
  load_ids(0, nit);
  wait_loads<0>();
  __syncthreads();
  next_item();
  for (int i = 0; i < S - 1; ++i) {
    issue_a(i);
    issue_b(i);
  }
  int slot = 0;
  for (int index = 0; index < n_items; ++index) {
    // no load beyond this item has been issued yet (nk >= S - 1)
    const ProductItem it = lit;
    const int live = max(0, min(C::MI, ((it.rows + 31) / 32 - wm + WM - 1) / WM));
    typename Acc<I8>::t32 acc[C::MI][C::NJ] = {};
    auto mma = [&](const Frag& f) {
#pragma unroll
      for (int m = 0; m < C::MI; ++m)
        if (m == 0 || m < live)
#pragma unroll
          for (int j = 0; j < C::NJ; ++j) acc[m][j] = mma32(f.b[j], f.a[m], acc[m][j]);
    };
    // one step's wait: the younger S - 2 steps may be in flight; then the loads of the step S - 1 ahead start
    auto begin_step = [&]() {
      wait_loads<(S - 2) * (C::NA + C::NB)>();
      __syncthreads();
      if (l_kb == nk && l_index + 1 < n_items) next_item();
    };
    if (live > 0) {
      // straight-line body: a branch around LDS reads would make the compiler wait for all of them at each use
      for (int kb = 0; kb < nk; ++kb) {
        begin_step();
        const u32x4* st = sm + slot * C::STAGE;
        const int to = slot == 0 ? S - 1 : slot - 1;
        Frag f[2];
        read_frags(f[0], st, 0);
        issue_a(to);
        read_frags(f[1], st, 1);
        mma(f[0]);
        issue_b(to);
#pragma unroll
        for (int s = 1; s < C::SUB; ++s) {
          if (s + 1 < C::SUB) read_frags(f[(s + 1) & 1], st, s + 1);
          mma(f[s & 1]);
        }
        slot = slot == S - 1 ? 0 : slot + 1;
      }
    } else {
      for (int kb = 0; kb < nk; ++kb) {
        begin_step();
        const int to = slot == 0 ? S - 1 : slot - 1;
        issue_a(to);
        issue_b(to);
        slot = slot == S - 1 ? 0 : slot + 1;
      }
    }
    // ---- epilogue
#pragma unroll
    for (int m = 0; m < C::MI; ++m) {
      const int r = (m * WM + wm) * 32;
      if (m >= live) break;
      const BlockRows br = {row_id(index, it, r + frow), row_id(index, it, r + (lane & 15)),
                            row_id(index, it, r + 16 + (lane & 15))};
      float sa = 1.0f;
      if constexpr (I8) sa = s_sa[(index & 1) * BM + r + frow];
      BlockAdd ad[C::NJ] = {};
      if constexpr (EPI) {
#pragma unroll
        for (int j = 0; j < C::NJ; ++j) ad[j] = load_add(p, br, it.n0 + (wn * C::NJ + j) * 32, lane);
      }
#pragma unroll
      for (int j = 0; j < C::NJ; ++j) {
        const int nl = (wn * C::NJ + j) * 32, at = (index & 1) * BN + nl;
        if (it.n0 + nl < p.N)
          store_block<I8, F32, EPI>(p, br, sa, s_sb + at, s_bias + at, ad[j], it.n0 + nl, lane, acc[m][j]);
      }
    }
  }
  wait_loads<0>();  // no load may reach LDS after the workgroup has ended
}

template <bool I8, bool F32, bool EPI, bool NT, bool TAIL, int BM, int BN, int WM, int WN, int S>
hipError_t ring_run(const ProductArgs& p, hipStream_t st) {
  using C = RingCfg<I8, EPI, BM, BN, WM, WN, S>;
  const auto kernel = ring_kernel<I8, F32, EPI, NT, TAIL, BM, BN, WM, WN, S>;
  // more than 64 KB of LDS has to be allowed once per device
  static std::atomic<uint64_t> allowed{0};
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(allowed.load(std::memory_order_relaxed) & bit)) {
    e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize,
                            (int)C::LDS);
    if (e != hipSuccess) return e;
    allowed.fetch_or(bit, std::memory_order_relaxed);
  }
  kernel<<<256 * C::PER_CU, C::NT, C::LDS, st>>>(p);
  return hipGetLastError();
}

// Rows that are whole steps, of which there are enough to fill the ring, and A offsets of 32 bits take the form
// without tail handling (grouped bf16 prefill 367 against 375 us with it).
template <bool I8, bool F32, bool EPI, bool NT, int BM, int BN, int WM, int WN, int S>
hipError_t ring_launch(const ProductArgs& p, hipStream_t st) {
  const int64_t a_rows = ((int64_t)p.R - 1) / p.a_div + 1;
  if (p.Kb % 128 == 0 && p.Kb / 128 >= S - 1 && a_rows * p.Kb <= ((int64_t)1 << 32))
    return ring_run<I8, F32, EPI, NT, false, BM, BN, WM, WN, S>(p, st);
  return ring_run<I8, F32, EPI, NT, true, BM, BN, WM, WN, S>(p, st);
}

ProductSize size_of(const ProductArgs& p) { return {p.P, p.R, p.E, p.N, p.Kb, p.off != nullptr}; }

template <bool I8, bool F32, bool EPI, bool NT>
hipError_t tiled_launch(const ProductArgs& p, hipStream_t st) {
  switch (product_tile(size_of(p), NT)) {
    case 0:
      if constexpr (!NT) return ring_launch<I8, F32, EPI, NT, 256, 256, 4, 2, 2>(p, st);
    case 1: return ring_launch<I8, F32, EPI, NT, 128, 256, 2, 4, 3>(p, st);
    case 2: return ring_launch<I8, F32, EPI, NT, 64, 128, 2, 2, 3>(p, st);
    case 3: return ring_launch<I8, F32, EPI, NT, 32, 128, 1, 4, 4>(p, st);
    default: return ring_launch<I8, F32, EPI, NT, 32, 64, 1, 2, 5>(p, st);
  }
}

template <bool F32, bool EPI>
hipError_t dense_i8_launch(const ProductArgs& p, hipStream_t st) {
  // The few-rows kernel against the best tile, us (rows x K x columns): 1 x 2048 x 4096 3.2 against 6.1, 16 rows 3.9
  // against 6.2; 33 x 512 x 4096 3.5 against 4.0, 64 x 1024 x 4096 4.6 against 4.8, 48 x 2048 x 4096 6.2 against 6.3,
  // 64 rows 7.3 against 6.5, 33 x 4096 x 4096 11.1 against 9.5 (every workgroup reads all rows of A, and its loads
  // come in batches).  256 workgroups fill the CUs.
  const unsigned blocks = (unsigned)((p.N + 15) / 16);
  if (p.P <= 16) {
    skinny_kernel<F32, EPI, 1, 4><<<blocks, 256, 0, st>>>(p);
    return hipGetLastError();
  }
  if (p.P <= 64 && p.Kb <= 2048 && p.P * p.Kb <= 48 * 2048 && blocks <= 256) {
    skinny_kernel<F32, EPI, 4, 2><<<blocks, 256, 0, st>>>(p);
    return hipGetLastError();
  }
  return tiled_launch<true, F32, EPI, false>(p, st);
}

template <bool I8, bool F32>
hipError_t grouped_launch(const ProductArgs& p, hipStream_t st) {
  if (product_streams(size_of(p))) return tiled_launch<I8, F32, false, true>(p, st);
  return tiled_launch<I8, F32, false, false>(p, st);
}

}  // namespace

hipError_t launch_product(const ProductArgs& args, bool i8, hipStream_t st) {
  ProductArgs p = args;
  // m = floor(2^(31 + l) / d) + 1 with l = ceil(log2 d): floor(id m / 2^(31 + l)) = floor(id / d) for id < 2^31
  if (p.a_div > 1) {
    int l = 1;
    while (l < 31 && (1u << l) < (unsigned)p.a_div) ++l;
    p.div_mul = (unsigned)((1ull << (31 + l)) / (unsigned)p.a_div + 1);
    p.div_shift = l - 1;
  }
  if (!i8) return p.c_f32 ? grouped_launch<false, true>(p, st) : grouped_launch<false, false>(p, st);
  if (p.off) return p.c_f32 ? grouped_launch<true, true>(p, st) : grouped_launch<true, false>(p, st);
  if (p.bias || p.add) return p.c_f32 ? dense_i8_launch<true, true>(p, st) : dense_i8_launch<false, true>(p, st);
  return p.c_f32 ? dense_i8_launch<true, false>(p, st) : dense_i8_launch<false, false>(p, st);
}

}  // namespace moe
