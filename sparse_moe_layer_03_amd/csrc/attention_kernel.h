// Attention of new tokens over a paged cache: the kernels, instantiated per type of the cache by attention_*.hip.
//
// Rows are (token, query head) pairs of one key head: row r of a sequence is token r / G, head r % G of the key head's
// G query heads, so that all of them read the key head's cache once.  Per 32 rows and 32 keys
//   S^T = K Q^T      lane l holds query row l & 31, keys 8 g + 4 (l >> 5) + i in register 4 g + i
//   O^T = V^T P^T    the same lanes hold the row's P, which the instruction takes as they are: its 16 keys a step are
//                    numbered 4 h + i and 8 + 4 h + i of lane half h, and V^T is read from LDS in that order,
//                    transposed by the LDS read itself
// so neither S nor P leaves its lane.  Softmax is the online form in base 2: running maximum m, sum l and O in fp32,
// rescaled when a tile raises m by more than 2^kSlack.  P is rounded to bf16 for its product, an error of the size of
// the output's own rounding (half a step, 2^-8 of each weight); where few rows leave the matrix cores idle the rest of
// it goes in as a second bf16 term (2^-16).  l sums the unrounded values.
//
// A masked key has P = 0, which does not undo an Inf or NaN in its V: rows behind the range of keys that the tile's
// rows can see are zeroed on the way into LDS, and in tiles with keys that only some rows see (later tokens, the
// window's edge) the values that are no numbers are, too.  These, behind all tiles, go to the rows that see them as
// they are: a weight is positive, and a sum with one holds an Inf or NaN whatever the weight and the rest.  A prompt of
// 4096, 8 heads over 1, takes 119 us, 117 with a NaN in an early value, 180 with one in every value.
//
// Three shapes.  Up to 32 rows a sequence (decoding, drafts): 32 rows, four waves that deal the keys out between them,
// K straight into the operand registers; the cache's bytes bound it.  64 requests of up to 8192 keys (4 heads of 128 in
// bf16, 537 MB) take 114 us, 4.7 TB/s, and 4.7 us to join, where the loads alone take 116 in all.  More rows: 128 rows
// in four waves that share tiles of 64 keys; with 512 such items of D 128 in bf16 256 rows in eight waves.  Bound
// between the matrix and the vector instructions: a prompt of 8192 tokens, 32 heads over 4, takes 531 to 554 us by the
// card, 993 to 1034 TFLOP/s of the 1487 that a large product reaches; of a wave's cycles the matrix instructions take
// 45%, the vector ones 40% (exponentials, maxima, rounding), LDS 28% without bank conflicts, and a third are waits.  At
// D 64 the exponentials weigh twice as much: 825 TFLOP/s.  Wide / narrow tiles, us: a prompt of 4096 148 / 163, two
// chunks of 1024 behind 8192 283 / 316, but one of 2048 (256 wide items) 68 / 59; at D 64, where three narrow workgroups
// fit a CU, a prompt of 8192 386 / 333.
//
// Measured and not taken, in us: two row blocks a wave (prefill 838 against 534, spills; D 64 312 against 328, but a
// window of 1024 91 against 80); tiles two deep in flight for 8-bit caches (no change); loads past the caches (decode
// 136 against 122); 256 workgroups instead of 512 at D up to 128 (decode 126 against 122, drafts 54 against 35); a
// wave's priority raised around its products, and the compiler's schedule groups (no change).
#pragma once

#include <atomic>

#include "attend_internal.h"
#include "attention_rule.h"

namespace moe {
namespace attn {

constexpr float kSlack = 8.0f;
constexpr float kNegInf = -__builtin_inff();

typedef short s16x4 __attribute__((ext_vector_type(4)));

// LDS by its own 32-bit addresses: constant distances become the instructions' offsets.
#define MOE_LDS __attribute__((address_space(3)))
typedef MOE_LDS unsigned char* lds_bytes;
template <class T>
__device__ __forceinline__ MOE_LDS T* lds_as(lds_bytes p) {
  return (MOE_LDS T*)p;
}
// A value that is worked out anew behind this point, not kept in a register from before a loop.
__device__ __forceinline__ int anew(int v) {
  asm volatile("" : "+v"(v));
  return v;
}

// D: head elements; CT: type of the cache; WR waves of 32 rows share a tile of KT keys; WK waves take every WK-th tile.
template <int D_, int CT_, int WR_, int WK_, int KT_>
struct Cfg {
  static constexpr int D = D_, CT = CT_, WR = WR_, WK = WK_, KT = KT_;
  static constexpr bool QUANT = CT != MOE_BF16;
  static constexpr int R = 32 * WR;            // rows of a workgroup
  static constexpr int UNIT = KT * WK;         // keys of a unit of work
  static constexpr int GT = 64 * WR;           // threads that load a tile
  static constexpr int THREADS = GT * WK;
  static constexpr int ROWB = D * (QUANT ? 1 : 2);
  static constexpr int CPR = ROWB / 16;        // 16-byte chunks of a cached row
  static constexpr int CHUNKS = KT * CPR;
  static constexpr int NL = (CHUNKS + GT - 1) / GT;
  static constexpr int NS = QUANT ? (2 * KT + GT - 1) / GT : 1;  // scales a thread loads
  static constexpr bool TWO = WR == 8;          // two groups of four waves, half a step apart
  static constexpr int NB = WR == 1 ? 1 : TWO ? 3 : 2;  // tiles in LDS: a wave alone needs no second one
  // Bytes from row to row in LDS, bf16.  A K read takes one 16-byte chunk of 32 rows: 16 rows in a row lie in different
  // banks.  A transposing V read takes four rows of 64 bytes, which do so likewise.
  static constexpr int KROW = 2 * D + 16, VROW = 2 * D + 64;
  static constexpr int SCALES = QUANT ? 2 * KT * 4 : 0;
  static constexpr bool KREG = WR == 1;  // K goes from memory into the operand registers
  static constexpr int KTILE = KREG ? 0 : KT * KROW;
  static constexpr int STAGE = (KTILE + KT * VROW > 32 * D * 4 || WK == 1 ? KTILE + KT * VROW : 32 * D * 4) + SCALES;
  // Page numbers a wave looks up per tile: of every load of whole rows, or of every 16 keys.  The 64 lanes of such a
  // load read rows that begin at a multiple of, and are at most, 16, so they lie in one page whatever its size.
  static constexpr int NP = KREG ? KT / 16 : NL;
  // q in LDS where it, O and the loads in flight would not fit the registers (spills wait behind those loads: 64 decode
  // requests at D 256 134 us, 151 with q in registers)
  static constexpr bool QLDS = KREG && D == 256 && !QUANT;
  static constexpr int SUMS = WK * NB * STAGE, QS = SUMS + (WK > 1 ? WK * 64 * 4 : 0);  // offsets in LDS
  static constexpr int ODD = QS + (QLDS ? 32 * KROW : 0);
  static constexpr int LDS = ODD + (WR > 1 ? 16 : 0);
  static constexpr int TERMS = WK > 1 ? 2 : 1;  // bf16 terms of P
  static constexpr int KB = KT / 32, NQ = D / 16, DB = D / 32;
  static_assert(WK == 1 || WR == 1, "");
  static_assert(!TWO || !QUANT, "the two groups' steps store no scales");
  static_assert(WK == 1 || STAGE >= 32 * D * 4, "the waves' O are merged in their tiles");
  static_assert(LDS <= 160 * 1024, "");
};

struct Seq {
  int q0, n, len;  // first row of q, new tokens, keys
};
// PTR: how q_start and kv_len are read, by lanes of their own or (s the same in all) by scalar loads.
typedef const __attribute__((address_space(4))) int32_t* scalar_ptr;
template <class PTR>
__device__ __forceinline__ Seq seq_at(const AttentionArgs& p, int s) {
  const PTR start = (PTR)(uintptr_t)p.q_start, len = (PTR)(uintptr_t)p.kv_len;
  Seq q;
  q.q0 = min(max(start[s], 0), p.T);
  q.n = max(min(max(start[s + 1], 0), p.T) - q.q0, 0);
  q.len = min(max(len[s], 0), p.max_pages << p.page_shift);
  return q;
}
// First key that any of the sequence's rows sees, down to a multiple of 64: where its units begin.
__device__ __forceinline__ int seq_base(const AttentionArgs& p, const Seq& q) {
  return p.window > 0 ? max(q.len - q.n - p.window + 1, 0) & ~63 : 0;
}
template <class C>
__device__ __forceinline__ int seq_units(const AttentionArgs& p, const Seq& q) {
  return max((q.len - seq_base(p, q) + C::UNIT - 1) / C::UNIT, 1);
}
template <class C>
__device__ __forceinline__ int row_tiles(const AttentionArgs& p, const Seq& q) {
  return (int)(((int64_t)q.n * p.G + C::R - 1) / C::R);
}
// Units of work of a sequence: all its row tiles and key heads times its keys.
template <class C, class PTR>
__device__ __forceinline__ int64_t seq_work(const AttentionArgs& p, int s) {
  const Seq q = seq_at<PTR>(p, s);
  return (int64_t)p.Hkv * row_tiles<C>(p, q) * seq_units<C>(p, q);
}

__device__ __forceinline__ int64_t wave_scan(int64_t v, int lane) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int64_t o = __shfl_up(v, d);
    if (lane >= d) v += o;
  }
  return v;
}
__device__ __forceinline__ int64_t lane_value(int64_t v, int lane) {
  const uint32_t lo = __builtin_amdgcn_readlane((int)v, lane), hi = __builtin_amdgcn_readlane((int)(v >> 32), lane);
  return (int64_t)((uint64_t)hi << 32 | lo);
}
// The sequence in which the running sum of weights passes `at`, and the sum before it; S if none does.  weight(s, PTR):
// of a sequence of the lane's own (const int32_t*) or the same in all (scalar_ptr).
template <class W>
__device__ __forceinline__ int find(int S, int lane, int64_t at, W weight, int64_t& before) {
  before = 0;
  if (S == 1) return at < weight(0, scalar_ptr()) ? 0 : 1;
  for (int b = 0; b < S; b += 64) {
    const int64_t incl = before + wave_scan(b + lane < S ? weight(b + lane, (const int32_t*)nullptr) : 0, lane);
    const int n = __popcll(__ballot(incl <= at));
    if (n < 64) {
      if (n > 0) before = lane_value(incl, n - 1);
      return b + n;
    }
    before = lane_value(incl, 63);
  }
  return S;
}
// Share `index` of `shares` equal ones (none below `least`) of all weights: its begin and end, and as `find` for its
// begin.
template <class W>
__device__ __forceinline__ int find_share(int S, int lane, int index, int shares, int least, W weight, int64_t& share,
                                          int64_t& begin, int64_t& end, int64_t& before) {
  int64_t total = 0, incl = 0;  // incl: of up to 64 sequences, one pass over them for both steps
  if (S == 1) {
    total = weight(0, scalar_ptr());
  } else {
    int64_t sum = 0;
    for (int b = 0; b < S; b += 64) sum += b + lane < S ? weight(b + lane, (const int32_t*)nullptr) : 0;
    incl = wave_scan(sum, lane);
    total = lane_value(incl, 63);
  }
  share = max((total + shares - 1) / shares, (int64_t)least);
  begin = index * share, end = min(total, begin + share);
  before = 0;
  if (S == 1 || begin >= end) return 0;
  if (S > 64) return find(S, lane, begin, weight, before);
  const int n = __popcll(__ballot(incl <= begin));
  if (n > 0) before = lane_value(incl, n - 1);
  return n;
}

// Scores and sums are kept by lane halves; both halves' maximum or sum.
__device__ __forceinline__ float halves_max(float v) {
  const auto x = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(x[0]), __uint_as_float(x[1]));
}
__device__ __forceinline__ float halves_sum(float v) {
  const auto x = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(x[0]) + __uint_as_float(x[1]);
}

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// Sixteen codes as two chunks of bf16 (every code is one exactly).
template <int CT>
__device__ __forceinline__ void widen(u32x4 w, u32x4& lo, u32x4& hi) {
  uint32_t o[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (CT == MOE_E4M3) {
      o[2 * i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[i], 1.0f, false));
      o[2 * i + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[i], 1.0f, true));
    } else {
      const int v = (int)w[i];
      o[2 * i] = cvt_bf16x2((float)(v << 24 >> 24), (float)(v << 16 >> 24));
      o[2 * i + 1] = cvt_bf16x2((float)(v << 8 >> 24), (float)(v >> 24));
    }
  }
  lo = u32x4{o[0], o[1], o[2], o[3]}, hi = u32x4{o[4], o[5], o[6], o[7]};
}

// Four elements of a cached row.
template <int CT>
__device__ __forceinline__ void cached4(const void* p, int64_t i, float* f) {
  if constexpr (CT == MOE_BF16) {
    const u32x2 w = *reinterpret_cast<const u32x2*>(static_cast<const uint16_t*>(p) + i);
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] = bf16_to_f32((uint16_t)(w[e >> 1] >> (16 * (e & 1))));
  } else {
    const uint32_t w = *reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(p) + i);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      f[e] = CT == MOE_I8 ? (float)((int)(w << (24 - 8 * e)) >> 24) : __builtin_amdgcn_cvt_f32_fp8(w >> (8 * e), 0);
  }
}
// The top bits of the elements of w that are no numbers (codes of int8 always are).
template <int CT>
__device__ __forceinline__ uint32_t odd_bits(uint32_t w) {
  if constexpr (CT == MOE_BF16) return ((w & 0x7f807f80u) + 0x00800080u) & 0x80008000u;
  if constexpr (CT == MOE_E4M3) return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
  return 0u;
}
__device__ __forceinline__ bool finite(float v) { return fabsf(v) < __builtin_inff(); }

// Partial results in the workspace: a Part per workgroup, then slots of R rows of O (unscaled, fp32) and R pairs
// (m, l).  Part w: the item that begins in workgroup w's share and ends behind it.
struct Part {
  int n;     // workgroups that hold a part of it, w the first; 0: there is no such item
  int rows;  // of the item
  int row0;  // its first, in the sequence's (token, head) rows
  int q0, h;
  int pos0;  // position of the sequence's token 0
  int none[2];
};
// A row's factor at the end: no key is seen, out 0; keys whose scores are all -infinity, 0 / 0.
__device__ __forceinline__ float inverse(float sum, int pos) {
  return sum > 0.0f || sum != sum ? 1.0f / sum : pos < 0 ? 0.0f : __builtin_nanf("");
}
template <class C>
__device__ __forceinline__ float* slot_at(const AttentionArgs& p, int slot) {
  return p.partial + (size_t)gridDim.x * (sizeof(Part) / 4) + (size_t)slot * C::R * (C::D + 2);
}

// One workgroup computes one (sequence, key head, row tile), or (STREAM) its equal share of all units of work, which
// may begin and end inside such an item: what is not a whole item goes to the workspace, slot 2 w for the end of an
// item and 2 w + 1 for a beginning, and combine_kernel joins it.  out may be q: this workgroup alone reads the q of a
// whole item, before it writes there, and what was cut is written in the next launch.
template <class C, bool STREAM>
__device__ __forceinline__ void attention_body(const AttentionArgs& p, int min_units, lds_bytes smem) {
  constexpr int D = C::D, KT = C::KT, WR = C::WR, WK = C::WK;
  constexpr bool KREG = C::KREG;
  const int lane0 = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wr = wave % WR, wk = wave / WR;

  const lds_bytes group = smem + wk * C::NB * C::STAGE;

  // Two words, for this item and the next: bits of tiles (tile_bit) that values were taken out of.
  MOE_LDS unsigned* const odd_tiles = lds_as<unsigned>(smem + C::ODD);
  int turn = 0;
  if constexpr (WR > 1) {
    if (threadIdx.x < 2) odd_tiles[threadIdx.x] = 0u;
    __syncthreads();
  }

  // ---- this workgroup's work
  int64_t u = 0, u_end = 1, before = 0, share = 1;
  int s, h = 0, m = 0;
  if constexpr (STREAM) {
    auto weight = [&](int i, auto ptr) { return seq_work<C, decltype(ptr)>(p, i); };
    s = find_share(p.S, lane0, blockIdx.x, gridDim.x, min_units, weight, share, u, u_end, before);
    // (written again below where there is such an item)
    if (threadIdx.x == 0) reinterpret_cast<Part*>(p.partial)[blockIdx.x].n = 0;
  } else {
    auto weight = [&](int i, auto ptr) { return (int64_t)row_tiles<C>(p, seq_at<decltype(ptr)>(p, i)); };
    // the last tiles, which see the most keys, first
    const int64_t tiles = gridDim.x / p.Hkv;
    h = blockIdx.x % p.Hkv;
    s = find(p.S, lane0, tiles - 1 - blockIdx.x / p.Hkv, weight, before);
    if (s >= p.S) return;
    m = (int)(tiles - 1 - blockIdx.x / p.Hkv - before);
  }

  while (u < u_end) {
    const Seq q = seq_at<scalar_ptr>(p, s);
    const int units = seq_units<C>(p, q), base = seq_base(p, q);
    int unit_lo = 0, unit_hi = units;
    if constexpr (STREAM) {
      const int tiles = row_tiles<C>(p, q);
      const int64_t work = (int64_t)p.Hkv * tiles * units;
      if (u >= before + work) {
        before += work;
        ++s;
        continue;
      }
      const int64_t at = u - before, item = at / units;
      unit_lo = (int)(at - item * units);
      unit_hi = (int)min((int64_t)units, unit_lo + (u_end - u));
      h = (int)(item / tiles), m = (int)(item - (int64_t)h * tiles);
    }
    const bool whole = unit_lo == 0 && unit_hi == units;
    if (WR > 1 && STREAM && threadIdx.x == 0) odd_tiles[turn ^ 1] = 0u;
    // ---- rows (what lanes derive from their number is not kept over the items: it would take some 40 registers)
    const int lane = anew(lane0), hh = lane >> 5, ql = lane & 31, gt = wr * 64 + lane;
    const int n_rows = q.n * p.G, r0 = m * C::R, wrow = r0 + wr * 32;
    const int pos0 = q.len - q.n;  // of token 0
    const int i_first = r0 / p.G, i_last = (min(r0 + C::R, n_rows) - 1) / p.G;
    // keys that the tile's rows see
    const int kb = p.window > 0 ? max(pos0 + i_first - p.window + 1, 0) : 0;
    const int ke = min(q.len, pos0 + i_last + 1);
    const bool wave_live = wrow < n_rows;
    const int w_lo = pos0 + min(wrow, n_rows - 1) / p.G, w_hi = pos0 + (min(wrow + 32, n_rows) - 1) / p.G;
    const int row = wrow + ql;
    const bool live = row < n_rows;
    const int tok = live ? row / p.G : 0, head = h * p.G + (live ? row - tok * p.G : 0);
    const int pos = live ? pos0 + tok : -1;
    const int vis0 = p.window > 0 ? max(pos - p.window + 1, 0) : 0, vis_n = max(pos - vis0 + 1, 0);

    bf16x8 qf[C::QLDS ? 1 : C::NQ];
    const lds_bytes ql_at = smem + C::QS + ql * C::KROW + 16 * hh;
    if constexpr (C::QLDS) {
      // the waves' rows are the same: each brings its share
      const uint16_t* qp = p.q + (q.q0 + tok) * p.q_ld + (int64_t)head * D + 8 * hh;
#pragma unroll
      for (int i = 0; i < C::NQ / WK; ++i) {
        u32x4 v = {0u, 0u, 0u, 0u};
        if (live) v = *reinterpret_cast<const u32x4*>(qp + 16 * (wk * (C::NQ / WK) + i));
        *lds_as<u32x4>(ql_at + 32 * (wk * (C::NQ / WK) + i)) = v;
      }
      __syncthreads();
    } else {
      // a K load of 16 codes is two steps' operand
      constexpr bool PAIRS = C::KREG && C::QUANT;
      const uint16_t* qp = p.q + (q.q0 + tok) * p.q_ld + (int64_t)head * D + (PAIRS ? 16 : 8) * hh;
#pragma unroll
      for (int i = 0; i < C::NQ; ++i) {
        u32x4 v = {0u, 0u, 0u, 0u};
        if (live) v = *reinterpret_cast<const u32x4*>(qp + (PAIRS ? 32 * (i / 2) + 8 * (i % 2) : 16 * i));
        qf[i] = __builtin_bit_cast(bf16x8, v);
      }
    }
    // ---- tiles: tile j of this wave's group begins at key_of(j)
    const int u_first = ke > kb ? max(unit_lo, (kb - base) / C::UNIT) : 0;
    const int u_last = ke > kb ? min(unit_hi, (ke - base + C::UNIT - 1) / C::UNIT) : 0;
    const int nt = max(u_last - u_first, 0);
    auto key_of = [&](int j) { return base + ((u_first + j) * WK + wk) * KT; };
    const scalar_ptr pages = (scalar_ptr)(uintptr_t)(p.pages + (int64_t)s * p.max_pages);
    const int page_mask = (1 << p.page_shift) - 1;
    // whether the workgroup's rows may differ in which of the tile's keys they see; such are among the first and the
    // last sixteen (256 rows are 256 tokens at most)
    auto mixed_tile = [&](int k0) {
      return k0 + KT - 1 > pos0 + i_first || (p.window > 0 && k0 <= pos0 + i_last - p.window);
    };
    auto tile_bit = [&](int j) { return nt - 1 - j < 16 ? nt - 1 - j : 16 + j; };
    unsigned odd = 0u;  // as odd_tiles, of a wave alone
    auto taken_out = [&](int j) {
      const unsigned bit = 1u << tile_bit(j);
      if constexpr (KREG)
        odd |= bit;
      else if (lane == 0)
        __hip_atomic_fetch_or(odd_tiles + turn, bit, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
    };
    // the page of a key, or of the nearest key that the rows see
    auto page_of = [&](int key) { return pages[min(max(key, kb), ke - 1) >> p.page_shift]; };

    u32x4 rk[C::NL], rv[C::NL];
    float rs[C::NS];
    auto first_row = [&](int i) { return KREG ? 16 * i : (i * C::GT + wr * 64) / C::CPR; };  // of page number i
    unsigned bad = 0;    // bit i: there is no such page
    int page[C::NP];     // of the next tile: a scalar load's latency ahead
    int64_t off[C::NP];  // of the tile at hand: where its rows begin in the cache, in bytes
    const uint32_t page_bytes = (uint32_t)p.Hkv * C::ROWB << p.page_shift;
    const uint32_t head_bytes = (uint32_t)h * C::ROWB << p.page_shift;
    auto look_up = [&](int j) {
      const int k0 = key_of(j);
#pragma unroll
      for (int i = 0; i < C::NP; ++i) page[i] = page_of(k0 + first_row(i));
    };
    auto find_rows = [&](int j) {
      const int k0 = key_of(j);
      bad = 0;
#pragma unroll
      for (int i = 0; i < C::NP; ++i) {
        const bool none = (unsigned)page[i] >= (unsigned)p.n_pages;
        bad |= none ? 1u << i : 0u;
        off[i] = (int64_t)((uint64_t)(none ? 0u : (unsigned)page[i]) * page_bytes) +
                 (head_bytes + (uint32_t)((k0 + first_row(i)) & page_mask) * C::ROWB);
      }
      if (j + 1 < nt) look_up(j + 1);
    };
    // Scales: a wave alone has the pages of all keys at hand; where more share a tile each lane looks up its own, a
    // tile ahead.
    int s_page[C::NS];
    auto scale_key = [&](int j, int i) { return key_of(j) + (i * C::GT + gt) % KT; };
    auto look_up_scales = [&](int j) {
      if constexpr (KREG) return;
#pragma unroll
      for (int i = 0; i < C::NS; ++i)
        s_page[i] = p.pages[(int64_t)s * p.max_pages + (min(max(scale_key(j, i), kb), ke - 1) >> p.page_shift)];
    };
    auto issue_scales = [&](int j) {
#pragma unroll
      for (int i = 0; i < C::NS; ++i) {
        const int x = i * C::GT + gt, key = scale_key(j, i);
        rs[i] = 0.0f;
        if constexpr (KREG) {
          const int g = x % KT >> 4;
          int64_t row = off[0];
#pragma unroll
          for (int n = 1; n < C::NP; ++n) row += g >= n ? off[n] - off[n - 1] : 0;
          if (x < 2 * KT && key >= kb && key < ke && !(bad >> g & 1))
            rs[i] = (x < KT ? p.k_scale : p.v_scale)[row / C::ROWB + (x & 15)];
        } else if (x < 2 * KT && key >= kb && key < ke && (unsigned)s_page[i] < (unsigned)p.n_pages) {
          const int64_t at = (((int64_t)s_page[i] * p.Hkv + h) << p.page_shift) + (key & page_mask);
          rs[i] = (x < KT ? p.k_scale : p.v_scale)[at];
        }
      }
      if (j + 1 < nt) look_up_scales(j + 1);
    };
    // rows as they lie, 64 chunks a load
    auto issue_rows = [&](const void* cache, u32x4* to, const int64_t* from) {
#pragma unroll
      for (int i = 0; i < C::NL; ++i) {
        if (C::CHUNKS % C::GT != 0 && i * C::GT + wr * 64 >= C::CHUNKS) break;
        const char* at = static_cast<const char*>(cache);
        if constexpr (C::KREG)
          at += from[i * 64 / C::CPR / 16] + (i * 64 / C::CPR % 16) * C::ROWB;
        else
          at += from[i];
        to[i] = *reinterpret_cast<const u32x4*>(at + (uint32_t)(lane * 16));
      }
    };
    // as the instruction takes K: lane l its key 32 b + (l & 31), chunk 2 i + (l >> 5)
    auto issue_k = [&]() {
#pragma unroll
      for (int b = 0; b < C::KB; ++b) {
        const char* at = static_cast<const char*>(p.k_cache);
        at += ql < 16 ? off[2 * b % C::NP] : off[(2 * b + 1) % C::NP];
        at += (ql & 15) * C::ROWB + 16 * hh;
#pragma unroll
        for (int i = 0; i < C::CPR / 2; ++i) rk[b * (C::CPR / 2) + i] = *reinterpret_cast<const u32x4*>(at + 32 * i);
      }
    };
    // this lane's place of load i
    const int c_lane = (wr * 64 + lane) % C::CPR, r_lane = (wr * 64 + lane) / C::CPR;
    // to LDS as bf16.  Rows outside the tile's range of keys become zeros; without a page (none: its bits) K becomes
    // NaN, and with it the scores of the rows that see it, V zeros.
    auto page_no = [&](int i) { return KREG ? i * 64 / C::CPR / 16 : i; };  // of load i
    auto store_rows = [&](u32x4* from, int j, lds_bytes to, int row_bytes, unsigned none, bool is_k) {
      const int k0 = key_of(j);
      const lds_bytes at = to + r_lane * row_bytes + c_lane * (C::QUANT ? 32 : 16);
      const bool edge = k0 < kb || k0 + KT > ke;
      constexpr int STEP = C::GT / C::CPR;  // rows from load to load
      if (edge || none) {
#pragma unroll
        for (int i = 0; i < C::NL; ++i) {
          const int key = k0 + r_lane + i * STEP;
          const bool out = key < kb || key >= ke, no_page = (none >> page_no(i) & 1) && !out;
          // codes have no NaN in all types: theirs is put in below
          const uint32_t v = no_page && is_k && !C::QUANT ? 0x7fc07fc0u : 0u;
          if (out || no_page) from[i] = u32x4{v, v, v, v};
        }
      }
      if (C::CT != MOE_I8 && !is_k && mixed_tile(k0)) {
        constexpr int TOP = C::QUANT ? 7 : 15;
        uint32_t bits = 0u;
#pragma unroll
        for (int i = 0; i < C::NL; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t b = odd_bits<C::CT>(from[i][e]);
            bits |= b, from[i][e] &= ~(b | (b - (b >> TOP)));
          }
        if (__any(bits != 0u)) taken_out(j);
      }
#pragma unroll
      for (int i = 0; i < C::NL; ++i) {
        if (C::CHUNKS % C::GT != 0 && i * C::GT + wr * 64 >= C::CHUNKS) break;
        MOE_LDS u32x4* t = lds_as<u32x4>(at + i * STEP * row_bytes);
        if constexpr (C::QUANT) {
          u32x4 lo, hi;
          widen<C::CT>(from[i], lo, hi);
          t[0] = lo, t[1] = hi;
        } else {
          t[0] = from[i];
        }
      }
      if (C::QUANT && is_k && none) {
#pragma unroll
        for (int i = 0; i < C::NL; ++i) {
          const int key = k0 + r_lane + i * STEP;
          if (C::CHUNKS % C::GT != 0 && i * C::GT + wr * 64 >= C::CHUNKS) break;
          if ((none >> page_no(i) & 1) && key >= kb && key < ke)
            lds_as<u32x4>(at + i * STEP * row_bytes)[0] = u32x4{0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u};
        }
      }
    };
    auto buf_v = [&](int buf) { return group + buf * C::STAGE + C::KTILE; };
    auto store_k = [&](int j, int buf, unsigned none) {
      store_rows(rk, j, group + buf * C::STAGE, C::KROW, none, true);
    };
    auto store_v = [&](int j, int buf, unsigned none) { store_rows(rv, j, buf_v(buf), C::VROW, none, false); };
    auto store_scales = [&](int j, int buf) {
      if (mixed_tile(key_of(j))) {
#pragma unroll
        for (int i = 0; i < C::NS; ++i) {
          const bool bad = i * C::GT + gt >= KT && !finite(rs[i]);
          if (__any(bad)) taken_out(j);
          if (bad) rs[i] = 0.0f;
        }
      }
      MOE_LDS float* ls = lds_as<float>(buf_v(buf) + KT * C::VROW);
#pragma unroll
      for (int i = 0; i < C::NS; ++i) {
        const int x = i * C::GT + gt;
        if (x < 2 * KT) ls[x] = x < KT ? rs[i] * p.scale : rs[i];
      }
    };

    f32x16 o[C::DB] = {};
    float mx = kNegInf, l = 0.0f;
    // whether this wave's rows see any key of the tile
    auto any_seen = [&](int k0) {
      return wave_live && k0 <= w_hi && k0 < ke && !(p.window > 0 && k0 + KT - 1 <= w_lo - p.window);
    };
    auto scores = [&](int buf, f32x16* x) {
      const lds_bytes lk = group + buf * C::STAGE + ql * C::KROW + hh * 16;
#pragma unroll
      for (int i = 0; i < C::NQ; ++i)
#pragma unroll
        for (int b = 0; b < C::KB; ++b)
          x[b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(*lds_as<bf16x8>(lk + 32 * b * C::KROW + 32 * i), qf[i], x[b],
                                                         0, 0, 0);
    };
    auto scores_k = [&](f32x16* x) {
#pragma unroll
      for (int b = 0; b < C::KB; ++b) {
#pragma unroll
        for (int i = 0; i < C::CPR / 2; ++i) {
          const u32x4 k = rk[b * (C::CPR / 2) + i];
          if constexpr (C::QUANT) {
            u32x4 lo, hi;
            widen<C::CT>(k, lo, hi);
            x[b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, lo), qf[2 * i], x[b], 0, 0, 0);
            x[b] =
                __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, hi), qf[2 * i + 1], x[b], 0, 0, 0);
          } else {
            bf16x8 f;
            if constexpr (C::QLDS)
              f = *lds_as<bf16x8>(ql_at + 32 * i);
            else
              f = qf[i];
            x[b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, k), f, x[b], 0, 0, 0);
          }
        }
        if (bad >> 2 * b & 3) {  // keys 32 b .. + 15 or + 16 .. + 31 have no page
#pragma unroll
          for (int e = 0; e < 16; ++e)
            if (bad >> (2 * b + (e >> 3)) & 1) x[b][e] = __builtin_nanf("");
        }
      }
    };
    const float scale = C::QUANT ? 1.0f : p.scale;  // 8-bit keys: in the scales
    auto scales_at = [&](int buf) { return lds_as<f32x4>(buf_v(buf) + KT * C::VROW + 16 * hh); };
    // masks the scores and brings m up to them
    auto maximum = [&](int k0, int buf, f32x16* x) {
      const bool masked = k0 + KT - 1 > w_lo || (p.window > 0 && k0 <= w_hi - p.window);
      if constexpr (C::QUANT) {
#pragma unroll
        for (int b = 0; b < C::KB; ++b)
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const f32x4 t = scales_at(buf)[8 * b + 2 * g];
#pragma unroll
            for (int i = 0; i < 4; ++i) x[b][4 * g + i] *= t[i];
          }
      }
      if (masked) {
#pragma unroll
        for (int b = 0; b < C::KB; ++b)
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const int key = k0 + 32 * b + 8 * (e >> 2) + 4 * hh + (e & 3);
            if ((unsigned)(key - vis0) >= (unsigned)vis_n) x[b][e] = kNegInf;
          }
      }
      float top = x[0][0];
#pragma unroll
      for (int b = 0; b < C::KB; ++b)
#pragma unroll
        for (int e = 0; e < 16; ++e) top = fmaxf(top, x[b][e]);
      top = halves_max(top) * scale;
      if (__any(top > mx + kSlack)) {
        const float to = top > mx + kSlack ? top : mx;  // a row's own need: its bits do not depend on its neighbours'
        const float f = exp2_fast(mx - (to == kNegInf ? 0.0f : to));
        mx = to;
        l *= f;
#pragma unroll
        for (int d = 0; d < C::DB; ++d) o[d] *= f;
      }
    };
    // scores to weights, as operands: hi[2 b + t], and what their rounding leaves in lo
    auto weights = [&](int buf, f32x16* x, u32x4* hi, u32x4* lo) {
      const float sub = mx == kNegInf ? 0.0f : mx;
      float sum[4] = {};
#pragma unroll
      for (int b = 0; b < C::KB; ++b)
#pragma unroll
        for (int t = 0; t < 2; ++t) {
#pragma unroll
          for (int e = 8 * t; e < 8 * t + 8; ++e) {
            x[b][e] = exp2_fast(fmaf(x[b][e], scale, -sub));
            sum[e & 3] += x[b][e];
          }
          if constexpr (C::QUANT) {
#pragma unroll
            for (int g = 2 * t; g < 2 * t + 2; ++g) {
              const f32x4 f = scales_at(buf)[KT / 4 + 8 * b + 2 * g];
#pragma unroll
              for (int i = 0; i < 4; ++i) x[b][4 * g + i] *= f[i];
            }
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float p0 = x[b][8 * t + 2 * i], p1 = x[b][8 * t + 2 * i + 1];
            const uint32_t w = cvt_bf16x2(p0, p1);
            hi[2 * b + t][i] = w;
            if constexpr (C::TERMS == 2)
              lo[2 * b + t][i] = cvt_bf16x2(p0 - __uint_as_float(w << 16), p1 - __uint_as_float(w & 0xffff0000u));
          }
        }
      l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
    };
    // O += P V
    auto product = [&](int buf, const u32x4* hi, const u32x4* lo) {
      const lds_bytes lv = buf_v(buf);
      // lane j of 16 reads row j / 4, elements 4 (j % 4) .. + 3, and gets element j of the four rows
      const lds_bytes tv = lv + (4 * hh + (lane >> 2 & 3)) * C::VROW + (lane >> 4 & 1) * 32 + (lane & 3) * 8;
#pragma unroll
      for (int b = 0; b < C::KB; ++b)
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const bf16x8 pf = __builtin_bit_cast(bf16x8, hi[2 * b + t]);
#pragma unroll
          for (int d = 0; d < C::DB; ++d) {
            const lds_bytes at = tv + (32 * b + 16 * t) * C::VROW + 64 * d;
            const s16x4 v0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16(lds_as<s16x4>(at));
            const s16x4 v1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16(lds_as<s16x4>(at + 8 * C::VROW));
            const auto v = __builtin_shufflevector(v0, v1, 0, 1, 2, 3, 4, 5, 6, 7);
            o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, v), pf, o[d], 0, 0, 0);
            if constexpr (C::TERMS == 2)
              o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, v),
                                                             __builtin_bit_cast(bf16x8, lo[2 * b + t]), o[d], 0, 0, 0);
          }
        }
    };
    // between LDS writes and reads of a tile: the waves that share it
    auto sync = [&]() {
      if constexpr (WR > 1)
        __syncthreads();
      else
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    };
    u32x4 hi[2 * C::KB], lo[2 * C::KB];
    if constexpr (C::KREG) {
      // a wave alone: the next tile is in flight from the end of this one's store on
      auto issue = [&](int j) {
        find_rows(j);
        issue_k();
        if constexpr (C::QUANT) issue_scales(j);
        issue_rows(p.v_cache, rv, off);
      };
      if (nt > 0) {
        look_up(0);
        if constexpr (C::QUANT) look_up_scales(0);
        issue(0);
      }
      for (int j = 0; j < nt; ++j) {
        const int k0 = key_of(j);
        f32x16 x[C::KB] = {};
        scores_k(x);
        sync();  // the last tile's reads are done
        if constexpr (C::QUANT) store_scales(j, 0);
        store_v(j, 0, bad);
        if (j + 1 < nt) issue(j + 1);
        sync();
        if (any_seen(k0)) {
          maximum(k0, 0, x);
          weights(0, x, hi, lo);
          product(0, hi, lo);
        }
      }
      sync();
    } else if (nt > 0) {
      // Scores run a tile ahead, so that their products and the exponentials of the tile before lie side by side.  Step
      // j: LDS holds K of tile j + 1 and V of tile j, K of j + 2 and V of j + 1 are in flight.
      int64_t v_off[C::NP];
      unsigned vbad = 0;
      auto next_k = [&](int j) {
        find_rows(j);
        issue_rows(p.k_cache, rk, off);
      };
      auto to_v = [&]() {  // V follows K by a tile
#pragma unroll
        for (int i = 0; i < C::NP; ++i) v_off[i] = off[i];
        vbad = bad;
      };
      auto next_v = [&](int j) {
        issue_rows(p.v_cache, rv, v_off);
        if constexpr (C::QUANT) issue_scales(j);
      };
      if constexpr (C::QUANT) look_up_scales(0);
      look_up(0);
      next_k(0), to_v(), next_v(0);
      store_k(0, 0, bad), store_v(0, 0, vbad);
      if constexpr (C::QUANT) store_scales(0, 0);
      if (nt > 1) {
        next_k(1);
        to_v(), next_v(1);
        store_k(1, 1, bad);
        if (nt > 2) next_k(2);
      }
      sync();
      f32x16 x[C::KB] = {};
      if (wave_live) scores(0, x);
      sync();
      if constexpr (C::TWO) {
        // Each SIMD has a wave of either group: one is at its matrix products (the scores of the next tile and this
        // tile's P V) while the other is at its exponentials, stores and loads; barriers keep them half a step apart.
        // Three tiles in LDS: what one group stores in its half no wave of the other still reads.
        int at = 0, next = 1, after = 2;
        const bool second = wr >= 4;
        if (second) sync();
        auto step = [&](int j, auto last) {
          if (wave_live) {
            maximum(key_of(j), at, x);
            weights(at, x, hi, lo);
          }
          if constexpr (!decltype(last)::value) {
            if (j + 2 < nt) store_k(j + 2, after, bad);
            store_v(j + 1, next, vbad);
            if (j + 2 < nt) to_v(), next_v(j + 2);
            if (j + 3 < nt) next_k(j + 3);
          }
          sync();
          if (wave_live) {
            if constexpr (!decltype(last)::value) {
#pragma unroll
              for (int b = 0; b < C::KB; ++b) x[b] = f32x16{};
              scores(next, x);
            }
            product(at, hi, lo);
          }
          sync();
          const int t = at;
          at = next, next = after, after = t;
        };
        for (int j = 0; j < nt - 1; ++j) step(j, std::false_type());
        step(nt - 1, std::true_type());
        if (!second) sync();
      } else {
        auto step = [&](int j, auto last) {
          const int buf = j & 1;
          if (wave_live) {
            maximum(key_of(j), buf, x);
            weights(buf, x, hi, lo);
            if constexpr (!decltype(last)::value) {
#pragma unroll
              for (int b = 0; b < C::KB; ++b) x[b] = f32x16{};
              scores(buf ^ 1, x);
            }
            product(buf, hi, lo);
          }
          if constexpr (!decltype(last)::value) {
            if (j + 2 < nt) store_k(j + 2, buf, bad);
            store_v(j + 1, buf ^ 1, vbad);
            if constexpr (C::QUANT) store_scales(j + 1, buf ^ 1);
            if (j + 2 < nt) to_v(), next_v(j + 2);
            if (j + 3 < nt) next_k(j + 3);
            sync();
          }
        };
        for (int j = 0; j < nt - 1; ++j) step(j, std::false_type());
        step(nt - 1, std::true_type());
      }
    }
    l = halves_sum(l);

    // ---- what was taken out of mixed tiles, to the rows that see it (behind the barrier after the last store)
    if constexpr (WR > 1) odd = __builtin_amdgcn_readfirstlane(odd_tiles[turn]), turn ^= 1;
    while (odd != 0u) {
      const int bit = __ffs(odd) - 1, k0 = key_of(bit < 16 ? nt - 1 - bit : bit - 16);
      odd &= odd - 1u;
#pragma unroll 1
      for (int key = max(k0, kb); key < min(k0 + KT, ke); ++key) {
        const int page = page_of(key);
        if ((unsigned)page >= (unsigned)p.n_pages) continue;  // (the scores of its rows are NaN)
        const int64_t at = (((int64_t)page * p.Hkv + h) << p.page_shift) + (key & page_mask);
        const float f = C::QUANT ? p.v_scale[at] : 1.0f;
        const bool seen = (unsigned)(key - vis0) < (unsigned)vis_n;
#pragma unroll
        for (int d = 0; d < C::DB; ++d)
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            float v[4];
            cached4<C::CT>(p.v_cache, at * D + 32 * d + 8 * g + 4 * hh, v);
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (seen && !(finite(v[e]) && finite(f))) o[d][4 * g + e] += v[e] * f;
          }
      }
    }

    // ---- to memory: blocks d0 .. d0 + nd - 1 of O (in v) of the lanes' rows
    const bool to_slot = STREAM && !whole;
    if (STREAM && unit_lo == 0 && !whole && threadIdx.x == 0) {
      const int64_t last = u + units - 1;  // the item's last unit
      reinterpret_cast<Part*>(p.partial)[blockIdx.x] = {(int)(last / share) - (int)blockIdx.x + 1,
                                                        min(n_rows - r0, C::R), r0, q.q0, h, pos0, {0, 0}};
    }
    float* slot = STREAM ? slot_at<C>(p, 2 * blockIdx.x + (unit_lo == 0 ? 1 : 0)) : nullptr;
    const int srow = wr * 32 + ql;  // row in the tile
    auto put4 = [&](int d, const float* v, float inv) {  // elements d .. d + 3
      if (to_slot) {
        *reinterpret_cast<float4*>(slot + (size_t)srow * D + d) = make_float4(v[0], v[1], v[2], v[3]);
      } else if (live) {
        *reinterpret_cast<u32x2*>(p.out + (q.q0 + tok) * p.out_ld + (int64_t)head * D + d) =
            u32x2{cvt_bf16x2(v[0] * inv, v[1] * inv), cvt_bf16x2(v[2] * inv, v[3] * inv)};
      }
    };
    auto put_sums = [&](float sm, float sl) {
      if (hh != 0) return;
      if (to_slot)
        *reinterpret_cast<float2*>(slot + (size_t)C::R * D + 2 * srow) = make_float2(sm, sl);
      else if (live && p.lse)
        p.lse[(int64_t)(q.q0 + tok) * p.Hq + head] =
            sl > 0.0f || sl != sl ? (sm + log2f(sl)) * 0.6931471805599453f : kNegInf;
    };
    if constexpr (WK == 1) {
      const float inv = inverse(l, pos);
      if (wave_live || to_slot) {
#pragma unroll
        for (int d = 0; d < C::DB; ++d)
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const float v[4] = {o[d][4 * g], o[d][4 * g + 1], o[d][4 * g + 2], o[d][4 * g + 3]};
            put4(32 * d + 8 * g + 4 * hh, v, inv);
          }
        put_sums(mx, l);
      }
      if (WR > 1 && STREAM) __syncthreads();  // before the next item's first tile
    } else {
      // the waves' results of the same rows joined: each adds its share of the elements of all
      MOE_LDS f32x2* ml = lds_as<f32x2>(smem + C::SUMS) + anew(ql);  // [WK][32]
      MOE_LDS float* mine = lds_as<float>(group) + anew(lane);                    // [16 DB][64]
      if (hh == 0) ml[wk * 32] = f32x2{mx, l};
      __syncthreads();
      float all = kNegInf, sum = 0.0f;
      f32x2 part[WK];
#pragma unroll
      for (int w = 0; w < WK; ++w) part[w] = ml[w * 32], all = fmaxf(all, part[w][0]);
      const float sub = all == kNegInf ? 0.0f : all;
#pragma unroll
      for (int w = 0; w < WK; ++w) sum += part[w][1] * exp2_fast(part[w][0] - sub);
      const float f = exp2_fast(mx - sub);
#pragma unroll
      for (int d = 0; d < C::DB; ++d)
#pragma unroll
        for (int e = 0; e < 16; ++e) mine[(16 * d + e) * 64] = o[d][e] * f;
      __syncthreads();
      const float inv = inverse(sum, pos);
      const int lane_at = anew(lane);
      constexpr int PER = C::DB * 4 / WK;  // groups of four registers a wave adds up
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int g4 = wk * PER + i;
        float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int w = 0; w < WK; ++w)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            v[e] += lds_as<float>(smem + w * C::NB * C::STAGE)[(4 * g4 + e) * 64 + lane_at];
        put4(32 * (g4 >> 2) + 8 * (g4 & 3) + 4 * hh, v, inv);
      }
      if (wk == 0) put_sums(all, sum);
      __syncthreads();  // before the next item's tiles
    }
    u += STREAM ? unit_hi - unit_lo : 1;
  }
}

template <class C, bool STREAM>
__global__ __launch_bounds__(C::THREADS, C::D == 256 ? 1 : 2) void attention_kernel(AttentionArgs p, int min_units) {
  extern __shared__ __align__(16) unsigned char smem[];
  attention_body<C, STREAM>(p, min_units, (lds_bytes)smem);
}

// ---- host
// Joins the partial results of the items that more than one workgroup computed; grid.x as in the launch before.  Up to
// FEW parts a row is a wave's, all its loads at once: 4.7 us for 64 requests, mostly the launch.  With more it is a
// workgroup's, its parts dealt over the waves: two rounds of loads, the parts' maxima and sums and then their O, 7.7 us
// for two contexts of 131072 (64 parts a row).
template <class C>
__global__ __launch_bounds__(256) void combine_kernel(AttentionArgs p) {
  constexpr int E = C::D / 64, MOST = 512, FEW = 8;
  __shared__ float weight[MOST], sums[4][C::D];
  const Part t = reinterpret_cast<const Part*>(p.partial)[blockIdx.x];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int first = (int)blockIdx.x;
  auto part = [&](int i) { return slot_at<C>(p, i == 0 ? 2 * first + 1 : 2 * (first + i)); };
  auto put = [&](int r, int d, float o, float inv) {
    const int row = t.row0 + r, tok = row / p.G, head = t.h * p.G + row - tok * p.G;
    p.out[(t.q0 + tok) * p.out_ld + (int64_t)head * C::D + d] = (uint16_t)cvt_bf16x2(o * inv, 0.0f);
  };
  auto put_lse = [&](int r, float top, float sum) {
    const int row = t.row0 + r, tok = row / p.G, head = t.h * p.G + row - tok * p.G;
    p.lse[(int64_t)(t.q0 + tok) * p.Hq + head] =
        sum > 0.0f || sum != sum ? (top + log2f(sum)) * 0.6931471805599453f : kNegInf;
  };
  const int rows = t.n > 0 ? t.rows : 0;
  if (t.n <= FEW) {
    // few parts: a row is a wave's
    for (int r = blockIdx.y * 4 + wave; r < rows; r += gridDim.y * 4) {
      float2 ml = make_float2(kNegInf, 0.0f);
      if (lane < t.n) ml = *reinterpret_cast<const float2*>(part(lane) + (size_t)C::R * C::D + 2 * r);
      float v[FEW][E];
#pragma unroll
      for (int i = 0; i < FEW; ++i)
        if (i < t.n)
#pragma unroll
          for (int e = 0; e < E; ++e) v[i][e] = part(i)[(size_t)r * C::D + lane + 64 * e];
      float top = ml.x;
#pragma unroll
      for (int d = 1; d < FEW; d <<= 1) top = fmaxf(top, __shfl_xor(top, d));
      top = __shfl(top, 0);
      const float f = exp2_fast(ml.x - (top == kNegInf ? 0.0f : top));
      const float sum = wave_sum(ml.y * f);
      float o[E] = {};
#pragma unroll
      for (int i = 0; i < FEW; ++i)
        if (i < t.n) {
          const float fi = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(f), i));
#pragma unroll
          for (int e = 0; e < E; ++e) o[e] += v[i][e] * fi;
        }
      const float inv = inverse(sum, t.pos0 + (t.row0 + r) / p.G);
#pragma unroll
      for (int e = 0; e < E; ++e) put(r, lane + 64 * e, o[e], inv);
      if (p.lse && lane == 0) put_lse(r, top, sum);
    }
    return;
  }
  for (int r = blockIdx.y; r < rows; r += gridDim.y) {
    float top = kNegInf, sum = 0.0f;
    float2 ml[MOST / 64];
#pragma unroll
    for (int i = 0; i < MOST / 64; ++i) {
      ml[i] = make_float2(kNegInf, 0.0f);
      if (i * 64 < t.n && i * 64 + lane < t.n)
        ml[i] = *reinterpret_cast<const float2*>(part(i * 64 + lane) + (size_t)C::R * C::D + 2 * r);
      top = fmaxf(top, ml[i].x);
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) top = fmaxf(top, __shfl_xor(top, d));
    const float sub = top == kNegInf ? 0.0f : top;
#pragma unroll
    for (int i = 0; i < MOST / 64; ++i) {
      const float f = exp2_fast(ml[i].x - sub);
      sum += ml[i].y * f;
      if (wave == 0 && i * 64 < t.n) weight[i * 64 + lane] = f;
    }
    sum = wave_sum(sum);
    __syncthreads();
    float v[E] = {};
#pragma unroll 8
    for (int i = wave; i < t.n; i += 4) {
      const float* a = part(i) + (size_t)r * C::D + lane * E;
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] += a[e] * weight[i];
    }
#pragma unroll
    for (int e = 0; e < E; ++e) sums[wave][lane * E + e] = v[e];
    __syncthreads();
    const float inv = inverse(sum, t.pos0 + (t.row0 + r) / p.G);
    if (threadIdx.x < C::D) {
      const int d = threadIdx.x;
      put(r, d, (sums[0][d] + sums[1][d]) + (sums[2][d] + sums[3][d]), inv);
    }
    if (p.lse && threadIdx.x == 0) put_lse(r, top, sum);
    __syncthreads();
  }
}

template <class C, bool STREAM>
hipError_t run(const AttentionArgs& a, const Plan& plan, hipStream_t st) {
  const auto kernel = attention_kernel<C, STREAM>;
  // more than 64 KB of LDS has to be allowed once per device
  static std::atomic<uint64_t> allowed{0};
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(allowed.load(std::memory_order_relaxed) & bit)) {
    e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, C::LDS);
    if (e != hipSuccess) return e;
    allowed.fetch_or(bit, std::memory_order_relaxed);
  }
  kernel<<<plan.grid, C::THREADS, C::LDS, st>>>(a, plan.min_units);
  if (STREAM && plan.grid > 1) combine_kernel<C><<<dim3(plan.grid, C::R / 4), 256, 0, st>>>(a);
  return hipGetLastError();
}

template <int D, int CT>
hipError_t run_type(const AttentionArgs& a, const Plan& plan, hipStream_t st) {
  using Few = Cfg<D, CT, 1, 4, D == 64 ? 64 : 32>;
  using Many = Cfg<D, CT, 4, 1, 64>;
  if (plan.rows == 32) return plan.stream ? run<Few, true>(a, plan, st) : run<Few, false>(a, plan, st);
  if constexpr (D == 128 && CT == MOE_BF16) {
    using Wide = Cfg<D, CT, 8, 1, 64>;
    if (plan.rows == 256) return run<Wide, false>(a, plan, st);
  }
  return plan.stream ? run<Many, true>(a, plan, st) : run<Many, false>(a, plan, st);
}

template <int CT>
hipError_t run_all(const AttentionArgs& a, const Plan& plan, hipStream_t st) {
  if (a.D == 64) return run_type<64, CT>(a, plan, st);
  if (a.D == 128) return run_type<128, CT>(a, plan, st);
  return run_type<256, CT>(a, plan, st);
}

hipError_t run_bf16(const AttentionArgs& a, const Plan& plan, hipStream_t st);
hipError_t run_i8(const AttentionArgs& a, const Plan& plan, hipStream_t st);
hipError_t run_e4m3(const AttentionArgs& a, const Plan& plan, hipStream_t st);

}  // namespace attn
}  // namespace moe
