// rb_tile.hpp -- a tile of a dense product on the matrix cores, and how a product's tiles are laid over the GPU.
//
//   out [M][N] = A [M][R] B,   B given as [N][R] (rows along the sum) or as [R][N] (columns along it), 16-bit operands,
//   fp32 sums; optionally two weight matrices side by side (their tiles' columns interleaved, so that one lane holds
//   both values of an output), or two products whose sums run on from one another.
//
// The kernels that use it own their epilogues: rb_glu.hip, rb_muon.hip.
#pragma once

#include <atomic>

#include "rb_elem.hpp"

namespace rb {
namespace tile {

typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef __bf16 b8 __attribute__((ext_vector_type(8)));
typedef float f4 __attribute__((ext_vector_type(4)));
typedef uint32_t u4 __attribute__((ext_vector_type(4)));
typedef short s4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) u4 lds_u4;
typedef __attribute__((address_space(3))) s4 lds_s4;
typedef __attribute__((address_space(3))) void lds_void;

__device__ __forceinline__ f4 mfma(_Float16, u4 a, u4 b, f4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8, a), __builtin_bit_cast(h8, b), c, 0, 0, 0);
}
__device__ __forceinline__ f4 mfma(__bf16, u4 a, u4 b, f4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(b8, a), __builtin_bit_cast(b8, b), c, 0, 0, 0);
}

// 16 bytes per lane from the buffer to LDS (lane l's at base + 16 l). The whole offset is the lane's, so that the
// range check sees all of it. Two forms of the same instruction: the compiler takes the transposing reads of LDS for
// dependent on every load to LDS in flight and has them wait for all of these (2048 x 4096 over 2 x 11008 in 411 us
// with the builtin), so where those reads are used the load is written out. It has no register outputs; its LDS writes
// are ordered by the kernel's own waits and barriers, as with the builtin. m0, where the LDS address goes, is an input of
// the statement, so that the compiler writes it and knows that it did (in the list of clobbers it is refused, being
// reserved). The waits in front: one state from the write of m0, five from a descriptor word that comes from a vector register.
template <bool kWritten> struct Rows {  // a buffer resource over [base, base + bytes)
  __amdgpu_buffer_rsrc_t r;
  Rows() = default;
  __device__ __forceinline__ Rows(const void* base, uint32_t bytes) : r(buffer_rsrc(base, bytes)) {}
  __device__ __forceinline__ void load(uint8_t* to, uint32_t off) const {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)to, 16, off, 0, 0, 0);
  }
};
template <> struct Rows<true> {
  u4 r;
  Rows() = default;
  __device__ __forceinline__ Rows(const void* base, uint32_t bytes) {
    const uint64_t p = reinterpret_cast<uint64_t>(base);
    r = (u4){(uint32_t)p, (uint32_t)(p >> 32) & 0xffffu, bytes, 0x00020000u};
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = __builtin_amdgcn_readfirstlane(r[i]);
  }
  __device__ __forceinline__ void load(uint8_t* to, uint32_t off) const {
    const uint32_t m0 = __builtin_amdgcn_readfirstlane((uint32_t)(size_t)(lds_void*)to);
    asm volatile("s_nop 4\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"{m0}"(m0), "v"(off), "s"(r) : "memory");
  }
};

constexpr int kTK = 64;            // terms of the sum per step
constexpr int kRowB = kTK * 2;     // bytes of a staged row along the sum
constexpr uint32_t kOob = 0x80000000u;
constexpr int kXcds = 8;
constexpr int kUnits = 256;        // compute units, and blocks of a full grid

// s_waitcnt immediates: vmcnt in bits 3:0 and 15:14, expcnt 6:4, lgkmcnt 11:8
constexpr int kWaitLds = 15 | (3 << 14) | (7 << 4);  // lgkmcnt = 0 alone
constexpr int wait_vmcnt(int n) { return (n & 15) | ((n >> 4) << 14) | (7 << 4) | (15 << 8); }

// One product: A rows along the sum; B, B2 as the tile's template says; R terms in `steps` steps of 64.
template <typename T>
struct Source {
  const T *A, *B, *B2;
  int64_t lda, ldb, ldb2;
  int R, steps;
};

// How `tiles` tiles of `steps` steps are laid over a grid of `grid` blocks (a multiple of 8). The first `full` of them
// are taken whole, in rounds of the grid; the next `cut` in runs of `chunk` steps, a block each, those of one run next
// to each other: the blocks of an XCD then pass the same steps at the same time and share what they load in
// its L2; the steps of the others in equal runs of `per` to all blocks, wherever these begin. Partial sums are joined by
// a second kernel: of a cut tile one for each run, of the others two partial tiles a block (its run starts in one
// tile and may end in the next).
struct Work {
  uint32_t tiles, tiles_m, full, cut, grid;
  int steps, chunk, per;
};
// the m and n of a tile: panels of 8 tiles along m, so that the 32 tiles that an XCD's units work on at a time
// share 8 blocks of A's rows and 4 of B's in its L2
__device__ __forceinline__ void place(uint32_t t, uint32_t tiles_m, uint32_t tiles, uint32_t& m, uint32_t& n) {
  const uint32_t tiles_n = tiles / tiles_m, panel = 8 * tiles_n, p = t / panel, r = t % panel;
  const uint32_t high = tiles_m - 8 * p < 8 ? tiles_m - 8 * p : 8;
  m = 8 * p + r % high;
  n = r / high;
}
// a block's number with the blocks of one XCD next to each other
__device__ __forceinline__ uint32_t block_of(uint32_t grid) { return blockIdx.x % kXcds * (grid / kXcds) + blockIdx.x / kXcds; }

// WM x WN waves, each TM x TN accumulators of v_mfma_f32_16x16x32: a tile of 16 WM TM rows by 16 WN TN columns. A step
// of 64 terms is one LDS stage of a ring of kS, and is two phases of 32 terms; a phase's fragments are read while
// the phase before it multiplies. In the middle of step s (the second phase's fragments are then in registers,
// so its stage is free) a wave waits for its own loads of step s + 1, the barrier makes everyone's visible, and
// the loads of step s + kS go into the freed stage.
//
// kNN: B is [R][N]; its fragments are read from LDS by the transposing read, whose 16 lanes take 4 rows by 16 columns.
// kHalf: of each wave's columns the first kHalf are B's and the others, for the same outputs, B2's; 0: B alone.
// kSrc: products whose sums run on from one another.
// kAl: rows of both operands are 16-byte aligned, R (and N where kNN) a multiple of 8: the rows go to LDS directly
// (buffer loads, which give 0 past a tile's rows and past the sum's end). Otherwise they pass through
// registers one step ahead, by 16-byte loads at any address.
template <typename T, int kWM, int kWN, int kTM, int kTN, int kS, bool kNN, int kHalf, int kSrc, bool kAl>
struct Tile {
  static constexpr int kWaves = kWM * kWN, kThreads = 64 * kWaves;
  static constexpr int BM = 16 * kWM * kTM, BN = 16 * kWN * kTN;       // staged rows of A and rows (columns) of B
  static constexpr int kOutN = kHalf ? BN / 2 : BN;                    // columns of the output
  static constexpr int kWaveN = kHalf ? kHalf : 16 * kTN;              // ... of one wave
  static constexpr int kStageA = BM * kRowB, kStage = kStageA + BN * kRowB;
  static constexpr int kPerA = BM / 8 / kWaves, kPerB = BN / 8 / kWaves, kPer = kPerA + kPerB;  // 1 KB groups per wave and step
  static constexpr int kRowNN = BN * 2;                                // bytes of a staged row of [R][N]
  static constexpr int kPad = 16 * kTN + 4;                            // floats of a row in the epilogue's LDS area
  static constexpr int kTurn = kWaves * 16 * kPad * 4;
  // Two stages of 256 x 256 leave room for half a stage: then an operand's part of a stage is a slot of its own, five of
  // them, which hold A and B of steps 0, 1, 2, ... in turn.
  static constexpr bool kFive = kAl && kS == 2 && kStageA * 2 == kStage && 5 * kStageA <= 160 * 1024;
  static constexpr int kSlots = kFive ? 5 * kStageA : kS * kStage;
  static constexpr int kLds = kSlots > kTurn ? kSlots : kTurn;
  static_assert(BM / 8 % kWaves == 0 && BN / 8 % kWaves == 0, "a load instruction has one operand");
  static_assert(kAl || kS == 2, "through registers a step is written two steps ahead");
  static_assert(!kHalf || (2 * kHalf == 16 * kTN && !kNN), "a wave holds both values of an output");
  static_assert(!kNN || BN == 256, "the transposing read's rows are 512 bytes");
  static_assert(kLds <= 160 * 1024, "LDS of a compute unit");

  static constexpr int kHalfN = kHalf;
  typedef f4 Acc[kTM][kTN];

  struct Where {
    int64_t m0;
    int n0, mrows, ncols;  // rows and columns that lie inside; n0, ncols count outputs
  };
  __device__ static __forceinline__ Where where(const Work& k, uint32_t t, int64_t M, int N) {
    uint32_t tm, tn;
    place(t, k.tiles_m, k.tiles, tm, tn);
    Where at;
    at.m0 = (int64_t)__builtin_amdgcn_readfirstlane(tm) * BM;
    at.n0 = (int)__builtin_amdgcn_readfirstlane(tn) * kOutN;
    at.mrows = M - at.m0 < BM ? (int)(M - at.m0) : BM;
    at.ncols = N - at.n0 < kOutN ? N - at.n0 : kOutN;
    return at;
  }

  // the sum's steps s0 .. s1 - 1 of the tile at `at` into acc. LDS is free for use before and after.
  __device__ static __forceinline__ void run(const Source<T> (&src)[kSrc], const Where& at, int N, int s0, int s1, uint8_t* smem,
                                             f4 (&acc)[kTM][kTN]) {
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int wm = w % kWM, wn = w / kWM;
    const int lr = lane & 15, lj = lane >> 4;

    // Rows along the sum: 1 KB groups of 8 rows; lane l fills slot l % 8 of row l / 8 with the 16-byte chunk
    // (l % 8) ^ (row % 8), so that the 8 rows of a fragment read's phase lie in 8 bank groups.
    // Rows of [R][N]: groups of 2 rows of 512 bytes; the 32-byte piece p of row k lies at p ^ ((k % 4) + 4 (k / 8 % 2)),
    // so that the 8 rows that 32 lanes of a transposing read take lie in 8 bank groups.
    const int xc = (lane & 7) ^ (lane >> 3);
    const int kr = lane >> 5;
    const int xn = (lane & 31) ^ (((2 * w + kr) & 3) | (w & 4)) * 2;
    const auto group_row = [&](int i) { return 8 * (i * kWaves + w); };  // of A, or of B with rows along the sum
    // B's rows: the wave that they belong to, which of two matrices, and the row counted in outputs
    const auto second = [&](int r) { return kHalf && (r / (kHalf ? kHalf : 1) & 1); };
    const auto out_row = [&](int r) { return kHalf ? r / (2 * kHalf) * kHalf + r % kHalf : r; };

    // the loads of a step's A or B to LDS at `base`: what they have in common, and the i-th of a wave
    struct Loads {
      Rows<kNN> r, r2;
      uint32_t v, v2, ld, ld2;
      bool ok;
      uint8_t* base;
    };
    const auto part_of = [&](int s, bool& next) -> const Source<T>& {
      next = kSrc == 2 && s >= src[0].steps;
      return src[kSrc == 2 && next ? kSrc - 1 : 0];
    };
    const auto loads_a = [&](int s, uint8_t* base) {
      bool next;
      const Source<T>& q = part_of(s, next);
      const int k0 = (next ? s - src[0].steps : s) * kTK;
      Loads l;
      l.ok = s < s1 && k0 + 8 * xc < q.R;
      l.base = base;
      l.ld = (uint32_t)q.lda * 2;
      l.r = Rows<kNN>(q.A + at.m0 * q.lda, (uint32_t)((at.mrows - 1) * (int)l.ld + q.R * 2));
      l.v = (uint32_t)(lane >> 3) * l.ld + 16u * xc + (uint32_t)k0 * 2;
      return l;
    };
    const auto loads_b = [&](int s, uint8_t* base) {
      bool next;
      const Source<T>& q = part_of(s, next);
      const int k0 = (next ? s - src[0].steps : s) * kTK;
      Loads l;
      l.ok = s < s1 && k0 + 8 * xc < q.R;
      l.base = base;
      l.ld = (uint32_t)q.ldb * 2;
      if constexpr (kNN) {
        const int rows = s < s1 ? q.R - k0 : 0;
        l.r = Rows<kNN>(q.B + (rows > 0 ? (int64_t)k0 * q.ldb : 0),
                          rows > 0 ? (uint32_t)(((rows < kTK ? rows : kTK) - 1) * (int)l.ld + N * 2) : 0u);
        l.v = (uint32_t)kr * l.ld + 16u * xn + (uint32_t)at.n0 * 2;
      } else {
        l.r = Rows<kNN>(q.B + (int64_t)at.n0 * q.ldb, (uint32_t)((at.ncols - 1) * (int)l.ld + q.R * 2));
        l.v = (uint32_t)(lane >> 3) * l.ld + 16u * xc + (uint32_t)k0 * 2;
        if constexpr (kHalf) {
          l.ld2 = (uint32_t)q.ldb2 * 2;
          l.r2 = Rows<kNN>(q.B2 + (int64_t)at.n0 * q.ldb2, (uint32_t)((at.ncols - 1) * (int)l.ld2 + q.R * 2));
          l.v2 = (uint32_t)(lane >> 3) * l.ld2 + 16u * xc + (uint32_t)k0 * 2;
        }
      }
      return l;
    };
    const auto load_a = [&](const Loads& l, int i) {
      l.r.load(l.base + (i * kWaves + w) * 1024, l.ok ? l.v + (uint32_t)group_row(i) * l.ld : kOob);
    };
    const auto load_b = [&](const Loads& l, int i) {
      uint8_t* const to = l.base + (i * kWaves + w) * 1024;
      if constexpr (kNN) {
        l.r.load(to, l.v + (uint32_t)(2 * (i * kWaves + w)) * l.ld);
      } else {
        const int r = group_row(i);
        if (second(r))
          l.r2.load(to, l.ok ? l.v2 + (uint32_t)out_row(r) * l.ld2 : kOob);
        else
          l.r.load(to, l.ok ? l.v + (uint32_t)out_row(r) * l.ld : kOob);
      }
    };
    const auto all_a = [&](int s, int at) {
      const Loads l = loads_a(s, smem + at);
#pragma unroll
      for (int i = 0; i < kPerA; ++i) load_a(l, i);
    };
    const auto all_b = [&](int s, int at) {
      const Loads l = loads_b(s, smem + at);
#pragma unroll
      for (int i = 0; i < kPerB; ++i) load_b(l, i);
    };

    // Through registers: a step's loads, all at addresses inside the rows (the vector that holds a row's end, and those
    // behind it, 8 elements before the end), so that none waits for another; when they are stored to LDS the vector at the
    // end is shifted and what lies behind the end becomes zero. Rows shorter than a vector are read by elements.
    u4 hold[kAl ? 1 : kPer];
    const bool short_n = kNN && N < 8;
    const auto fetch = [&](int s, u4 (&hold)[kAl ? 1 : kPer]) {
      const bool next = kSrc == 2 && s >= src[0].steps;
      const Source<T>& q = src[kSrc == 2 && next ? kSrc - 1 : 0];
      const int k0 = (next ? s - src[0].steps : s) * kTK, c = k0 + 8 * xc;
      const int ca = c < q.R - 8 ? c : q.R - 8, col = at.n0 + 8 * xn, cb = col < N - 8 ? col : N - 8;
      const auto rows = [&](auto load_k, auto load_n) {  // load_k(row): along the sum; load_n(row): across it
#pragma unroll
        for (int i = 0; i < kPerA; ++i) {  // a row past the last one repeats it: its outputs are not stored
          const int r = group_row(i) + (lane >> 3);
          hold[i] = load_k(q.A + (at.m0 + (r < at.mrows ? r : at.mrows - 1)) * q.lda);
        }
#pragma unroll
        for (int i = 0; i < kPerB; ++i) {
          if constexpr (kNN) {
            const int k = k0 + 2 * (i * kWaves + w) + kr;
            hold[kPerA + i] = load_n(q.B + (int64_t)(k < q.R ? k : q.R - 1) * q.ldb);
          } else {
            const int g = group_row(i), r = out_row(g) + (lane >> 3);
            const int64_t n = at.n0 + (r < at.ncols ? r : at.ncols - 1);
            hold[kPerA + i] = load_k(second(g) ? q.B2 + n * q.ldb2 : q.B + n * q.ldb);
          }
        }
      };
      const auto vec = [](const T* p) { return __builtin_bit_cast(u4, *reinterpret_cast<const typename Vec8<T>::Raw*>(p)); };
      const auto few = [](const T* row, int c, int n) { return __builtin_bit_cast(u4, load8<T>(row, c, n)); };
      if (q.R >= 8 && !short_n)
        rows([&](const T* row) { return vec(row + ca); }, [&](const T* row) { return vec(row + cb); });
      else
        rows([&](const T* row) { return few(row, c, q.R); }, [&](const T* row) { return few(row, col, N); });
    };
    const auto put = [&](int s, int stage, const u4 (&hold)[kAl ? 1 : kPer]) {
      const bool next = kSrc == 2 && s >= src[0].steps;
      const Source<T>& q = src[kSrc == 2 && next ? kSrc - 1 : 0];
      const int k0 = (next ? s - src[0].steps : s) * kTK, c = k0 + 8 * xc, col = at.n0 + 8 * xn;
      const bool ends_k = k0 + kTK > q.R, ends_n = kNN && at.n0 + BN > N;  // uniform
      const bool by_elements = q.R < 8 || short_n;
      const auto fix = [&](u4 v, int c, int n) {
        if (by_elements) return v;
        typename Vec8<T>::Raw r = __builtin_bit_cast(typename Vec8<T>::Raw, v);
        shift_down(r, 8 - n % 8);
        const u4 t = __builtin_bit_cast(u4, r), zero = {0, 0, 0, 0};
        return c + 8 <= n ? v : c < n ? t : zero;
      };
      const auto store = [&](auto value) {
#pragma unroll
        for (int i = 0; i < (kAl ? 1 : kPer); ++i)
          *reinterpret_cast<u4*>(smem + stage * kStage + (i < kPerA ? 0 : kStageA) +
                                 ((i < kPerA ? i : i - kPerA) * kWaves + w) * 1024 + lane * 16) = value(i);
      };
      if (!ends_k && !ends_n) {
        store([&](int i) { return hold[i]; });
      } else {
        store([&](int i) {
          if (!kNN || i < kPerA) return fix(hold[i], c, q.R);
          const bool past = k0 + 2 * ((i - kPerA) * kWaves + w) + kr >= q.R;
          return past ? (u4){0, 0, 0, 0} : fix(hold[i], col, N);
        });
      }
    };

#pragma unroll
    for (int i = 0; i < kTM; ++i)
#pragma unroll
      for (int j = 0; j < kTN; ++j) acc[i][j] = (f4){0.f, 0.f, 0.f, 0.f};

    const uint32_t lds0 = (uint32_t)(size_t)(__attribute__((address_space(3))) uint8_t*)smem;
    const uint32_t f0 = lr * kRowB + 16u * ((uint32_t)lj ^ (lr & 7u)), f1 = lr * kRowB + 16u * ((4u + lj) ^ (lr & 7u));
    const uint32_t aa = lds0 + wm * kTM * 16 * kRowB;
    const uint32_t ab = lds0 + (kNN ? (8 * lj + (lr >> 2)) * kRowNN + 8 * (lr & 3) : wn * kTN * 16 * kRowB);
    const uint32_t turn_nn = (lr >> 2) | (lj & 1) << 2;
    u4 xf[2][kTM], wf[2][kTN];
    constexpr int kReads = kTM + kTN, kProducts = kTM * kTN;
    constexpr int kReadSpan = kProducts < 2 * kReads ? kProducts : kProducts / 2;  // products that the reads are spread over
    const auto read_one = [&](int kh, int in_a, int in_b, int r) {  // the r-th fragment of half kh of the step whose A and B lie there
      if (r >= kTN) {
        xf[kh][r - kTN] = *(lds_u4*)(size_t)(aa + in_a + (r - kTN) * 16 * kRowB + (kh ? f1 : f0));
      } else if constexpr (kNN) {
        const uint32_t p = ab + in_b + kh * 32 * kRowNN + 32 * (((uint32_t)(wn * kTN + r)) ^ turn_nn);
        const s4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4*)(size_t)p);
        const s4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4*)(size_t)(p + 4 * kRowNN));
        wf[kh][r] = __builtin_bit_cast(u4, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
      } else {
        wf[kh][r] = *(lds_u4*)(size_t)(ab + in_b + r * 16 * kRowB + (kh ? f1 : f0));
      }
    };
    // The products of half kh with the reads of the other half (of the step that lies at in_a, in_b) and the wave's loads
    // among them, in this order: the compiler takes a load to LDS and a read of LDS for dependent and would put all of one before the other,
    // and the products behind both. Issued together, the loads of 8 waves hold each wave up until the memory pipeline
    // has taken them, 16 cycles each.
    const auto phase = [&](int kh, int in_a, int in_b, int loads, auto load) {
#pragma unroll
      for (int p = 0; p < kProducts; ++p) {
        const int i = p / kTN, j = p % kTN;
        acc[i][j] = mfma(T(0), wf[kh][j], xf[kh][i], acc[i][j]);
#pragma unroll
        for (int r = p * kReads / kReadSpan; r < (p + 1) * kReads / kReadSpan && r < kReads; ++r) read_one(kh ^ 1, in_a, in_b, r);
#pragma unroll
        for (int l = p * loads / kProducts; l < (p + 1) * loads / kProducts; ++l) load(l);
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    const auto barrier = [] {  // the raw barrier: __syncthreads would also wait for every load in flight
      asm volatile("" ::: "memory");
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
    };

    // where A and B of a step lie: slots 2 s and 2 s + 1 (mod 5) from s0 on, or the stages of the ring
    const auto bump = [](int x, int by) { return x + by >= kSlots ? x + by - kSlots : x + by; };
    constexpr int kStep = kFive ? 2 * kStageA : kStage;
    int in_a = 0, in_b = kStageA;
    if constexpr (kFive) {
      all_a(s0, 0), all_b(s0, kStageA), all_a(s0 + 1, 2 * kStageA), all_b(s0 + 1, 3 * kStageA), all_a(s0 + 2, 4 * kStageA);
      __builtin_amdgcn_s_waitcnt(wait_vmcnt(2 * kPerA + kPerB));
    } else if constexpr (kAl) {
#pragma unroll
      for (int s = 0; s < kS; ++s) all_a(s0 + s, s * kStage), all_b(s0 + s, s * kStage + kStageA);
      __builtin_amdgcn_s_waitcnt(wait_vmcnt((kS - 1) * kPer));
    } else {
      u4 ahead[kAl ? 1 : kPer];
      fetch(s0, hold);
      fetch(s0 + 1, ahead);
      put(s0, 0, hold);
      put(s0 + 1, 1, ahead);
      fetch(s0 + 2, hold);
      __builtin_amdgcn_s_waitcnt(kWaitLds);
    }
    barrier();
#pragma unroll
    for (int r = 0; r < kReads; ++r) read_one(0, in_a, in_b, r);
    __builtin_amdgcn_sched_barrier(0);
    for (int s = s0; s < s1; ++s) {
      phase(0, in_a, in_b, 0, [](int) {});
      const int free_a = in_a, free_b = in_b;
      in_a = bump(in_a, kStep), in_b = bump(in_b, kStep);
      __builtin_amdgcn_s_waitcnt(kFive ? wait_vmcnt(kPerA) & kWaitLds : kAl ? wait_vmcnt((kS - 2) * kPer) & kWaitLds : kWaitLds);
      barrier();
      if constexpr (kFive) {
        // five slots: B of step s + 2 goes where A of step s was, A of step s + 3 where its B was, so that half of what
        // the next wait is for has been on its way for two steps
        const Loads lb = loads_b(s + 2, smem + free_a), la = loads_a(s + 3, smem + free_b);
        __builtin_amdgcn_sched_barrier(0);
        phase(1, in_a, in_b, kPer, [&](int i) { i < kPerB ? load_b(lb, i) : load_a(la, i - kPerB); });
      } else if constexpr (kAl) {
        const Loads la = loads_a(s + kS, smem + free_a), lb = loads_b(s + kS, smem + free_b);
        __builtin_amdgcn_sched_barrier(0);
        phase(1, in_a, in_b, kPer, [&](int i) { i < kPerA ? load_a(la, i) : load_b(lb, i - kPerA); });
      } else {
        put(s + 2, free_a / kStage, hold);
        fetch(s + 3, hold);
        __builtin_amdgcn_sched_barrier(0);
        phase(1, in_a, in_b, 0, [](int) {});
      }
    }
    // loads past the last step (out of range, zeros) end before LDS is used again
    __builtin_amdgcn_s_waitcnt(wait_vmcnt(0));
    __syncthreads();
  }

  // The accumulators by rows: 16 rows at a time through the wave's own LDS area, so that consecutive lanes hold
  // consecutive columns and whole lines are read and written. f(row, column, p): the tile's row, the output column
  // counted from n0 (a multiple of 8), and p[0 .. 7] its fp32 sums (p[kHalf .. kHalf + 7] the second matrix's), which it
  // may change. D of the product: lane l holds columns 4 (l / 16) .. + 3 of row l % 16. turned(row, column, p) is called
  // once for 16 rows and all of the wave's columns and sees what f left (row stride kPad). LDS must be free; the block
  // synchronises before its next use.
  // ahead(s, row, column) is called before the 16 rows are turned, for what f will read at the s-th of its kPasses places.
  static constexpr int kLanes = kWaveN / 8, kAtOnce = 64 / kLanes, kPasses = 16 / kAtOnce;  // lanes of a row, rows at once
  template <typename A, typename F, typename G>
  __device__ static __forceinline__ void rows_ahead(const f4 (&acc)[kTM][kTN], uint8_t* smem, A ahead, F f, G turned) {
    walk(acc, smem, ahead, [&](int i, int w, int lane, float* turn) {
#pragma unroll
      for (int s = 0; s < kPasses; ++s) pass(i, s, w, lane, turn, f);
    }, turned);
  }
  template <typename F, typename G>
  __device__ static __forceinline__ void rows(const f4 (&acc)[kTM][kTN], uint8_t* smem, F f, G turned) {
    walk(acc, smem, [](int, int, int) {}, [&](int i, int w, int lane, float* turn) {
#pragma unroll 1
      for (int s = 0; s < kPasses; ++s) pass(i, s, w, lane, turn, [&](int, int r, int c, float* p) { f(r, c, p); });
    }, turned);
  }

 private:
  template <typename F>
  __device__ static __forceinline__ void pass(int i, int s, int w, int lane, float* turn, F f) {
    const int r = kAtOnce * s + lane / kLanes, c = 8 * (lane % kLanes);
    f(s, ((w % kWM) * kTM + i) * 16 + r, (w / kWM) * kWaveN + c, turn + r * kPad + c);
  }
  template <typename A, typename P, typename G>
  __device__ static __forceinline__ void walk(const f4 (&acc)[kTM][kTN], uint8_t* smem, A ahead, P passes, G turned) {
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int lr = lane & 15, lj = lane >> 4;
    float* const turn = reinterpret_cast<float*>(smem) + w * (16 * kPad);
#pragma unroll 1
    for (int i = 0; i < kTM; ++i) {
#pragma unroll
      for (int s = 0; s < kPasses; ++s)
        pass(i, s, w, lane, turn, [&](int s, int r, int c, float*) { ahead(s, r, c); });
#pragma unroll
      for (int q = 0; q < kTM; ++q)
        if (q == i) {
#pragma unroll
          for (int j = 0; j < kTN; ++j) *reinterpret_cast<f4*>(turn + lr * kPad + 16 * j + 4 * lj) = acc[q][j];
        }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      passes(i, w, lane, turn);
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      turned(((w % kWM) * kTM + i) * 16, (w / kWM) * kWaveN, turn);
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
  }
};

__device__ __forceinline__ void eight(const float* p, float (&v)[8]) {
  const f4 lo = *reinterpret_cast<const f4*>(p), hi = *reinterpret_cast<const f4*>(p + 4);
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = lo[j], v[4 + j] = hi[j];
}

// A block's share of the work, tile by tile: body(tile, first step, end step, slot): slot -1 for a whole tile, else the
// partial tile in the workspace that takes the sums.
template <typename F>
__device__ __forceinline__ void share(const Work& k, F body) {
  const uint32_t lb = block_of(k.grid);
  const uint32_t rest = k.tiles - k.full - k.cut;
  uint32_t t = lb, it = lb * (uint32_t)k.per, slot = k.grid + 2 * lb;
  bool cut = k.cut > 0 && (int64_t)(lb / k.cut) * k.chunk < k.steps;
  const uint32_t all = rest * (uint32_t)k.steps;
  const uint32_t end = it + (uint32_t)k.per < all ? it + (uint32_t)k.per : all;
  for (;;) {
    uint32_t tile = t;
    int s0 = 0, s1 = k.steps, to = -1;
    if (t < k.full) {
      t += k.grid;
    } else if (cut) {
      cut = false;
      tile = k.full + lb % k.cut;
      s0 = (int)(lb / k.cut) * k.chunk;
      if (k.steps - s0 > k.chunk) s1 = s0 + k.chunk;
      to = (int)lb;
    } else if (it < end) {
      const uint32_t q = it / (uint32_t)k.steps;
      tile = k.full + k.cut + q;
      s0 = (int)(it - q * (uint32_t)k.steps);
      if (k.steps - s0 > (int)(end - it)) s1 = s0 + (int)(end - it);
      to = (int)slot++;
      it += (uint32_t)(s1 - s0);
    } else {
      break;
    }
    body(tile, s0, s1, to);
  }
}

// The partial tiles of split tile q (counted from `full`), in the order of the sum: f(slot) for each.
template <typename F>
__device__ __forceinline__ void parts(const Work& k, uint32_t q, F f) {
  if (q < k.cut) {
    for (int s0 = 0; s0 < k.steps; s0 += k.chunk, q += k.cut) f(q);
    return;
  }
  const uint32_t a = (q - k.cut) * (uint32_t)k.steps, b = a + (uint32_t)k.steps, per = (uint32_t)k.per;
  for (uint32_t lb = a / per; lb * per < b; ++lb) f(k.grid + 2 * lb + (lb * per < a ? 1 : 0));
}

// The rest of a product's tiles that does not fill a round of the grid is split where that is estimated to take less
// time than one more round: into as many equal runs each as there are blocks for, or into one run more where that leaves
// some of the tiles over, whose steps are then shared by all. A run is 4 steps at least; a split costs its partial
// tiles' way to memory and back (5 MB / us) and 4 us for the second launch; a tile's ends cost 4 us; a step that is not shared in the L2 costs half
// as much again. `step`: us of one step when every unit works.
struct Lay {
  Work work;
  double est;
  size_t part_bytes;  // of the partial tiles
};
inline Lay lay(int64_t tiles_m, int64_t tiles_n, int64_t steps, double step, int64_t tile_bytes) {
  const int64_t tiles = tiles_m * tiles_n, rounds = tiles / kUnits, rest = tiles % kUnits;
  const auto eights = [](int64_t n) { return (uint32_t)((n + kXcds - 1) / kXcds * kXcds); };
  Lay l{};
  l.work.tiles = (uint32_t)tiles, l.work.tiles_m = (uint32_t)tiles_m, l.work.steps = (int)steps;
  l.work.full = (uint32_t)tiles;
  l.work.grid = rounds > 0 ? (uint32_t)kUnits : eights(rest);
  constexpr double kTile = 4.0;  // us of a tile's beginning and end
  l.est = 3.0 + (double)(rounds + (rest > 0)) * ((double)steps * step + kTile);
  if (rest == 0 || rest * steps >= (int64_t)1 << 31) return l;
  const int64_t most = (steps + 3) / 4 > 1 ? (steps + 3) / 4 : 1;  // runs of a tile
  for (int64_t runs = kUnits / rest; runs <= kUnits / rest + 1; ++runs) {
    if (runs < 2 || runs > most) {
      if (runs < 2 || kUnits / rest < most) continue;
      runs = most;  // few tiles of few steps: not every unit gets a run
      if (runs < 2) break;
    }
    const int64_t chunk = (steps + runs - 1) / runs, each = (steps + chunk - 1) / chunk;
    const int64_t cut = each * rest <= kUnits ? rest : kUnits / each, left = rest - cut;
    const int64_t per = (left * steps + kUnits - 1) / kUnits;
    if (chunk >= steps || cut < 1 || per >= steps) break;
    const int64_t blocks = left > 0 || rounds > 0 ? kUnits : eights(cut * each);
    const int64_t kept = left > 0 ? 3 * blocks : cut * each, moved = 2 * (cut * each + (left > 0 ? kUnits + left : 0));
    const double est = 7.0 + (double)rounds * ((double)steps * step + kTile) + (double)chunk * step + kTile +
                       (left > 0 ? (double)per * 1.5 * step + kTile : 0.0) + (double)(moved * tile_bytes) / 5e6;
    if (est < l.est) {
      l.work.full = (uint32_t)(tiles - rest), l.work.cut = (uint32_t)cut, l.work.chunk = (int)chunk;
      l.work.per = (int)per, l.work.grid = (uint32_t)blocks;
      l.est = est, l.part_bytes = (size_t)(kept * tile_bytes);
    }
    if (runs == most) break;
  }
  return l;
}

// Lets a kernel take `bytes` of dynamic LDS on the current device; `done` holds a bit for every device where it may.
template <typename K>
hipError_t allow_lds(std::atomic<uint64_t>& done, K kernel, int bytes) {
  int device = 0;
  if (const hipError_t e = hipGetDevice(&device); e != hipSuccess) return e;
  const uint64_t bit = device < 64 ? uint64_t(1) << device : 0;
  if (done.load(std::memory_order_relaxed) & bit) return hipSuccess;
  const hipError_t e = hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == hipSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

inline bool rows16(const void* p, int64_t ld) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && ld % 8 == 0; }
inline bool lines(const void* p, int64_t ld, int size) { return reinterpret_cast<uintptr_t>(p) % 128 == 0 && ld * size % 128 == 0; }

}  // namespace tile
}  // namespace rb
