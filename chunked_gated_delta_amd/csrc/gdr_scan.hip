// The sequential part of the head-gated delta rule: the state from chunk to chunk, and the outputs.
//
// Value columns are independent, so a workgroup owns one (sequence, value head) and 16 of its columns and
// walks the chunks:
//   E = V - gam K S  |  U = beta T' E  |  S <- e^{G_last} S + K^T (eta U)         O = scale gam Q S + P U
// with a barrier at each bar.  What bounds it is that chain: three products of 16 columns, each waiting
// for the one before, so everything else is kept off it.
//  - Wavefronts 0-3 walk the chain.  Wavefront i owns token rows 16i .. 16i + 15 and a quarter of the
//    state's rows, in registers (fp32 matrix-core results).  Wavefronts 4-7, one more on each SIMD, form the
//    outputs (or, in the backward's run, write out the entering states and F) in the chain's shadow.
//  - Every A operand (K, Q, K^T, T', P) has exactly one reader in the workgroup and is loaded straight into its
//    registers, the chain's kAhead chunks ahead, as soon as the registers' present contents are used.  Loads
//    past the last chunk are clamped to it.
//  - What the wavefronts exchange (the state, E, U: 16 columns each) goes through LDS as ready B operands.
//  - The compute unit's address path is what limits a step next (77 % busy when each lane fetched its own
//    values of v and the gates and wrote its own of o), so wavefronts 4-7 move v, o and the gates in
//    rows of 16 bytes a lane and turn them in LDS.
// Rows behind the sequence's end read its last row; their E is set to zero, so nothing of them reaches
// the state, and their outputs are not written.
#include <type_traits>

#include "gdr_internal.h"

namespace kda {

namespace {

constexpr int kAhead = 2;   // chunks ahead that the chain's operands are loaded

__device__ __forceinline__ int64_t min64(int64_t a, int64_t b) { return a < b ? a : b; }
__device__ __forceinline__ float value(uint16_t x) { return bf16_to_f32(x); }
__device__ __forceinline__ float value(float x) { return x; }

// Writes `rows` contraction places x 16 NT columns of B operands (first planes; `tile` bytes from one column
// tile to the next) to row-major memory: a lane takes 8 columns of one place.
template <typename T, int NT>
__device__ __forceinline__ void write_rows(const char* frags, int frag_bytes, int tile, int rows, GlobalPtr<T> out, int ld, int tid) {
  for (int i = tid; i < rows * 2 * NT; i += 256) {
    const int r = i / (2 * NT), c0 = (i & 1) * 8, nt = (i >> 1) % NT;
    const char* fr = frags + nt * tile + (r >> 5) * frag_bytes;
    T x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = frag_at<T>(fr, r & 31, c0 + e);
    typename Frags<T>::In v;
    __builtin_memcpy(&v, x, sizeof(v));
    *repoint<typename Frags<T>::In>(out + r * ld + 16 * nt + c0) = v;
  }
}

// All ones or zeros, of a condition on values of the wavefront.  Positions advance by masked amounts, not
// behind a branch, which would come between matrix instructions and the reads of their results (see settle).
__device__ __forceinline__ int64_t mask_of(bool c) { return __builtin_amdgcn_readfirstlane(c ? -1 : 0); }

// Byte offsets, from a chunk's first row, of the rows that a lane reads of a strided tensor: row `row` as
// an A operand, rows r0 .. r0 + 3 as part of a result tile; in the last chunk the rows behind the
// sequence's end become its last one.
struct LaneRow {
  uint32_t whole, tail;
  __device__ __forceinline__ LaneRow(int row, int last_rows, int64_t stride, int at, int esz)
      : whole((uint32_t)((row * stride + at) * esz)), tail((uint32_t)((min(row, last_rows - 1) * stride + at) * esz)) {}
  __device__ __forceinline__ uint32_t of(bool last) const { return last ? tail : whole; }
};

// 64 tokens x 16 NT columns in LDS, column by column (a result tile's lane reads 4 tokens of its column).
// 128 NT threads move them: thread t has 8 columns of token t / (2 NT).
template <typename T, int NT> struct Turned {
  static constexpr int kLd = sizeof(T) == 2 ? 72 : 68, kPer = 2 * NT;
  T x[16 * NT * kLd];
  __device__ __forceinline__ void put_row(int t, const typename Frags<T>::In& v) {
    T e8[8];
    __builtin_memcpy(e8, &v, sizeof(v));
#pragma unroll
    for (int e = 0; e < 8; ++e) x[(8 * (t % kPer) + e) * kLd + t / kPer] = e8[e];
  }
  __device__ __forceinline__ typename Frags<T>::In row(int t) const {
    T e8[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) e8[e] = x[(8 * (t % kPer) + e) * kLd + t / kPer];
    typename Frags<T>::In v;
    __builtin_memcpy(&v, e8, sizeof(v));
    return v;
  }
  __device__ __forceinline__ floatx4 tile(int col, int r0) const {
    if constexpr (sizeof(T) == 2) {
      const u32x2v p = *reinterpret_cast<const u32x2v*>(x + col * kLd + r0);
      return floatx4{lo_bf16(p[0]), hi_bf16(p[0]), lo_bf16(p[1]), hi_bf16(p[1])};
    } else {
      return *reinterpret_cast<const floatx4*>(x + col * kLd + r0);
    }
  }
  __device__ __forceinline__ void put_tile(int col, int r0, floatx4 v) {
    if constexpr (sizeof(T) == 2) *reinterpret_cast<u32x2v*>(x + col * kLd + r0) = u32x2v{pk_bf16(v[0], v[1]), pk_bf16(v[2], v[3])};
    else *reinterpret_cast<floatx4*>(x + col * kLd + r0) = v;
  }
};
// a chunk's gates in LDS
struct Gates {
  float gam[64], eta[64], beta[64];
};

template <typename T, int DK, int NT, bool STATES>
__global__ __launch_bounds__(512) void gdr_scan_kernel(GdrParams p) {
  using In = typename Frags<T>::In;
  using Op3 = typename Frags<T>::template Op<3>;
  using Op2 = typename Frags<T>::template Op<2>;
  constexpr int KS = DK / 32;
  constexpr int RT = DK >= 64 ? DK / 64 : 1;      // state row tiles of a wavefront
  constexpr int kOp1 = op_frag<T, 1>(), kOp2 = op_frag<T, 2>(), kOp3 = op_frag<T, 3>();
  __shared__ __attribute__((aligned(16))) char sf[NT][KS * kOp3];          // the state, as B operands
  __shared__ __attribute__((aligned(16))) char ef[NT][2 * kOp3];           // E
  __shared__ __attribute__((aligned(16))) char wf[NT][2 * kOp3];           // eta U
  __shared__ __attribute__((aligned(16))) char uf[NT][2 * kOp2];           // U (F where states are written)
  __shared__ __attribute__((aligned(16))) Rows<T, DK> kl;                  // the chunk's K
  __shared__ __attribute__((aligned(16))) Turned<T, NT> vt[2];             // v, by the chunk's parity
  __shared__ __attribute__((aligned(16))) Turned<T, NT> ot;                // o on its way out
  __shared__ __attribute__((aligned(16))) Gates gate[2];

  int64_t unit;
  int part;
  if (!gdr_block(blockIdx.x, p.n_seq * p.Hv, p.dv / (16 * NT), &unit, &part)) return;
  const int64_t s = unit / p.Hv;
  const int h = (int)(unit % p.Hv), kh = h / (p.Hv / p.Hk);
  const GdrSeq seq = gdr_seq(p, s);
  const int64_t nc = seq.n_chunks;
  const int lane = threadIdx.x & 63, li = lane & 15, g = lane >> 4;
  const int wave = wave_id() & 3;
  const int col0 = 16 * NT * part;                // first of the workgroup's columns
  const int r0 = 16 * wave + 4 * g;               // first of this lane's 4 token rows in result tiles
  const int last_rows = (int)(seq.len - (nc - 1) * kGdrChunk);   // tokens of the last chunk
  const int64_t blk0 = seq.slot0 * p.Hv + h;      // workspace block of chunk 0; the next is Hv further
  const auto gates = global_in<float>(p.ws_gate) + blk0 * kGateFloats;

  if (wave_id() < 4) {
    const bool owner = wave * RT < DK / 16;
    floatx4 S[NT][RT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int m = 0; m < RT; ++m) {
        S[nt][m] = floatx4{};
        if (owner && p.S0) {
          const auto at = global_in<float>(p.S0) + unit * p.dk * p.dv + (16 * (wave * RT + m) + 4 * g) * p.dv + col0 + 16 * nt + li;
#pragma unroll
          for (int r = 0; r < 4; ++r) S[nt][m][r] = at[r * p.dv];
        }
      }
    auto put_state = [&]() {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int m = 0; m < RT; ++m) {
          const int t = wave * RT + m;
          if (owner) put_op<3>(sf[nt] + (t >> 1) * kOp3, t & 1, li, g, S[nt][m], T{});
        }
    };
    put_state();
    block_barrier();

    // BOTH: the wavefront's rows of T' reach into both steps of 32 tokens (wavefronts 2 and 3)
    auto walk = [&](auto both) {
      constexpr int TS = decltype(both)::value ? 2 : 1;
      struct Buf {
        In k[KS];
        Op3 ti[TS];
      };
      // where the next loads come from
      int64_t at = 0;
      auto kp = global_in<T>(p.k) + seq.row * p.sk.b + kh * p.sk.h + seq.t0 * p.sk.t;
      auto tp = as_global((const char*)p.ws_ti) + blk0 * kTriFrags * kOp3 + lower_frag(wave, 0) * kOp3;
      const LaneRow krow(16 * wave + li, last_rows, p.sk.t, 8 * g, sizeof(T));
      auto load_k = [&](Buf& b) {
        const auto from = lane_at(kp, krow.of(at == nc - 1));
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) b.k[ks] = load_row8(from + 32 * ks);
      };
      auto load_ti = [&](Buf& b) {   // and on to the next chunk
#pragma unroll
        for (int ks = 0; ks < TS; ++ks) b.ti[ks] = load_frag<Op3>(tp + ks * kOp3, lane);
        const int64_t more = mask_of(at < nc - 1);
        at += more & 1;
        kp += more & (int64_t)(kGdrChunk * p.sk.t);
        tp += more & (int64_t)(p.Hv * (kTriFrags * kOp3));
      };
      auto step = [&](Buf& b, int64_t c, int n) {
        const Gates& gt = gate[c & 1];
        const floatx4 gam = ld4f((const float*)gt.gam + r0);
        floatx4 E[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          Op3 sb[KS];
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) sb[ks] = load_frag<Op3>((const char*)sf[nt] + ks * kOp3, lane);
          E[nt] = mma_steps(b.k, sb, floatx4{});
        }
        // K also goes to LDS, for the transpose; rows behind the end meet zeros of eta U
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) kl.put8(16 * wave + li, 32 * ks + 8 * g, b.k[ks]);
        load_k(b);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const floatx4 v = vt[c & 1].tile(16 * nt + li, r0);
#pragma unroll
          for (int r = 0; r < 4; ++r) E[nt][r] = r0 + r < n ? v[r] - gam[r] * E[nt][r] : 0.f;
          put_op<3>(ef[nt] + (wave >> 1) * kOp3, wave & 1, li, g, E[nt], T{});
        }
        block_barrier();

        const floatx4 eta = ld4f((const float*)gt.eta + r0), beta = ld4f((const float*)gt.beta + r0);
        floatx4 F[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          Op3 eb[TS];
#pragma unroll
          for (int ks = 0; ks < TS; ++ks) eb[ks] = load_frag<Op3>((const char*)ef[nt] + ks * kOp3, lane);
          F[nt] = mma_steps(b.ti, eb, floatx4{});
        }
        load_ti(b);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) put_op<3>(wf[nt] + (wave >> 1) * kOp3, wave & 1, li, g, eta * (beta * F[nt]), T{});
        block_barrier();

        In kt[RT][2];
        const int first = owner ? wave * RT : 0;
#pragma unroll
        for (int m = 0; m < RT; ++m)
#pragma unroll
          for (int ks = 0; ks < 2; ++ks) kt[m][ks] = kl.transposed(first + m, ks, lane);
        const float last = gt.gam[63];   // e^{G_last}: tokens behind the end do not decay
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const Op3 wb[2] = {load_frag<Op3>((const char*)wf[nt], lane), load_frag<Op3>((const char*)wf[nt] + kOp3, lane)};
          put_op<2>(uf[nt] + (wave >> 1) * kOp2, wave & 1, li, g, STATES ? F[nt] : beta * F[nt], T{});
#pragma unroll
          for (int m = 0; m < RT; ++m) S[nt][m] = mma_steps(kt[m], wb, S[nt][m] * last);
        }
        put_state();
        block_barrier();
      };
      if (nc > 0) {
        Buf buf[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          load_k(buf[i]);
          load_ti(buf[i]);
        }
        int64_t c = 0;
        for (; c + kAhead < nc; c += kAhead) {
#pragma unroll
          for (int i = 0; i < kAhead; ++i) step(buf[i], c + i, kGdrChunk);
        }
        if (kAhead > 1 && c + 1 < nc) {
          step(buf[0], c, kGdrChunk);
          step(buf[kAhead - 1], c + 1, last_rows);
        } else {
          step(buf[0], c, last_rows);
        }
      }
    };
    static_assert(kAhead == 1 || kAhead == 2, "the loop's remainder");
    if (wave < 2) walk(std::false_type{});
    else walk(std::true_type{});
    if constexpr (!STATES) block_barrier();   // the last chunk's outputs, between wavefronts 4-7
    if (p.S_final && owner) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int m = 0; m < RT; ++m) {
          const auto at = global_out<float>(p.S_final) + unit * p.dk * p.dv + (16 * (wave * RT + m) + 4 * g) * p.dv + col0 + 16 * nt + li;
#pragma unroll
          for (int r = 0; r < 4; ++r) at[r * p.dv] = S[nt][m][r];
        }
    }
    return;
  }

  // v and the gates of one chunk ahead of the chain: loaded, then left in LDS
  const int tid = threadIdx.x & 255;
  constexpr int kPer = 2 * NT;                    // threads to a token's columns
  In vx;
  float gx = 0.f;
  int64_t ahead = 0;
  auto vp = global_in<T>(p.v) + seq.row * p.sv.b + h * p.sv.h + seq.t0 * p.sv.t + col0;
  auto gp = gates + (wave < 3 ? wave : 0) * 64;
  static_assert(kGateGam == 0 && kGateEta == 64 && kGateBeta == 128, "a wavefront each");
  const LaneRow vrow(tid / kPer, last_rows, p.sv.t, 8 * (tid % kPer), sizeof(T));
  auto fetch = [&]() {
    if (wave < kPer) vx = load_row8(lane_at(vp, vrow.of(ahead == nc - 1)));
    if (wave < 3) gx = *lane_at(gp, lane * 4);
    const int64_t more = mask_of(ahead < nc - 1);
    ahead += more & 1;
    vp += more & (int64_t)(kGdrChunk * p.sv.t);
    gp += more & (int64_t)(p.Hv * kGateFloats);
  };
  auto leave = [&](int64_t c) {
    if (wave < kPer) vt[c & 1].put_row(tid, vx);
    if (wave < 3) (wave == 0 ? gate[c & 1].gam : wave == 1 ? gate[c & 1].eta : gate[c & 1].beta)[lane] = gx;
  };
  if (nc > 0) {
    fetch();
    leave(0);
    fetch();
  }
  block_barrier();   // the first state, v and gates
  if constexpr (STATES) {
    auto sp = global_out<T>(p.ws_s) + blk0 * p.dk * p.dv + col0;
    auto fp = global_out<T>(p.ws_f) + blk0 * kGdrChunk * p.dv + col0;
    for (int64_t c = 0; c < nc; ++c) {
      // the state that enters this chunk, F of the one before
      write_rows<T, NT>(sf[0], kOp3, KS * kOp3, DK, sp, p.dv, tid);
      sp += p.Hv * (p.dk * p.dv);
      if (c > 0) {
        write_rows<T, NT>(uf[0], kOp2, 2 * kOp2, kGdrChunk, fp, p.dv, tid);
        fp += p.Hv * (kGdrChunk * p.dv);
      }
      block_barrier();
      leave(c + 1);
      fetch();
      block_barrier();
      block_barrier();
    }
    if (nc > 0) write_rows<T, NT>(uf[0], kOp2, 2 * kOp2, kGdrChunk, fp, p.dv, tid);
  } else {
    auto op = global_out<T>(p.o) + seq.row * p.so.b + h * p.so.h + seq.t0 * p.so.t + col0;
    const uint32_t orow = (uint32_t)(((tid / kPer) * p.so.t + 8 * (tid % kPer)) * sizeof(T));
    auto store = [&](int n) {
      if (tid < kPer * n) *repoint<In>(lane_at(op, orow)) = ot.row(tid);
      op += kGdrChunk * p.so.t;
    };
    auto walk = [&](auto both) {
      constexpr int TS = decltype(both)::value ? 2 : 1;
      struct Buf {
        In q[KS], pm[TS];
      };
      int64_t at = 0;
      auto qp = global_in<T>(p.q) + seq.row * p.sq.b + kh * p.sq.h + seq.t0 * p.sq.t;
      auto pp = as_global((const char*)p.ws_p) + blk0 * kTriFrags * kOp1 + lower_frag(wave, 0) * kOp1;
      const LaneRow qrow(16 * wave + li, last_rows, p.sq.t, 8 * g, sizeof(T));
      auto load = [&](Buf& b) {
        const auto from = lane_at(qp, qrow.of(at == nc - 1));
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) b.q[ks] = load_row8(from + 32 * ks);
#pragma unroll
        for (int ks = 0; ks < TS; ++ks) b.pm[ks] = load_frag<In>(pp + ks * kOp1, lane);
        const int64_t more = mask_of(at < nc - 1);
        at += more & 1;
        qp += more & (int64_t)(kGdrChunk * p.sq.t);
        pp += more & (int64_t)(p.Hv * (kTriFrags * kOp1));
      };
      floatx4 O[NT];
      // the outputs of the chunk before, whose U the chain has left; two planes of U and of the state, as o is
      // rounded to the inputs' type
      auto add_own = [&](Buf& b) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          Op2 ub[TS];
#pragma unroll
          for (int ks = 0; ks < TS; ++ks) ub[ks] = load_frag<Op2>((const char*)uf[nt] + ks * kOp2, lane);
          O[nt] = mma_steps(b.pm, ub, O[nt]);
        }
      };
      // outputs from the chunk's entering state; meanwhile the chunk before is finished
      auto step = [&](Buf& b, Buf& before, int64_t c) {
        if (c > 0) add_own(before);
        const floatx4 gam = ld4f((const float*)gate[c & 1].gam + r0);
        floatx4 read[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          Op2 sb[KS];
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) sb[ks] = load_frag<Op2>((const char*)sf[nt] + ks * kOp3, lane);
          read[nt] = mma_steps(b.q, sb, floatx4{});
          settle(read[nt]);
        }
        block_barrier();
        if (c > 0) {
          load(before);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) ot.put_tile(16 * nt + li, r0, O[nt]);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) O[nt] = (p.scale * gam) * read[nt];
        leave(c + 1);
        fetch();
        block_barrier();
        if (c > 0) store(kGdrChunk);
        block_barrier();
      };
      if (nc > 0) {
        Buf b0, b1;
        load(b0);
        load(b1);
        int64_t c = 0;
        for (; c + 1 < nc; c += 2) {
          step(b0, b1, c);
          step(b1, b0, c + 1);
        }
        if (c < nc) {
          step(b0, b1, c);
          add_own(b0);
        } else {
          add_own(b1);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) ot.put_tile(16 * nt + li, r0, O[nt]);
      }
    };
    if (wave < 2) walk(std::false_type{});
    else walk(std::true_type{});
    block_barrier();
    if (nc > 0) store(last_rows);
  }
}

// The adjoint's sequential part, from the last chunk to the first, in the same division of work:
//   X = P^T dO + eta K dS  |  dU = T^T X, dE = beta dU (the gradient of v)
//   |  dS <- e^{G_last} dS + Q^T (scale gam dO) - K^T (gam dE)
// Wavefronts 0-3 walk the chain; wavefronts 4-7 form P^T dO and Q^T (scale gam dO) of the chunk that comes
// next, which do not depend on it, and write out dS of each chunk's end for the gradient kernel.  The
// chain leaves, per 16 columns, the sums of dU F that make beta's gradient.
template <typename T, int DK, int NT>
__global__ __launch_bounds__(512) void gdr_rscan_kernel(GdrParams p) {
  using In = typename Frags<T>::In;
  using Op3 = typename Frags<T>::template Op<3>;
  constexpr int KS = DK / 32;
  constexpr int RT = DK >= 64 ? DK / 64 : 1;
  constexpr int kIn = in_frag<T>(), kOp3 = op_frag<T, 3>();
  constexpr int kPer = 2 * NT;                    // threads to a token's columns
  __shared__ __attribute__((aligned(16))) char sf[NT][KS * kOp3];          // dS
  __shared__ __attribute__((aligned(16))) char xf[NT][2 * kOp3];           // X
  __shared__ __attribute__((aligned(16))) char ef[NT][2 * kOp3];           // -gam dE
  __shared__ __attribute__((aligned(16))) char of[NT][2 * kIn];            // dO
  __shared__ __attribute__((aligned(16))) char gf[NT][2 * kOp3];           // scale gam dO
  __shared__ __attribute__((aligned(16))) float x0[NT][4 * 256];           // P^T dO, result tiles [wave][lane][4]
  __shared__ __attribute__((aligned(16))) float d0[NT][DK / 16 * 256];     // Q^T (scale gam dO)
  __shared__ __attribute__((aligned(16))) Rows<T, DK> kl, ql;              // the chain's K, the next chunk's Q
  __shared__ __attribute__((aligned(16))) Turned<T, NT> ot;                // dO on its way in
  __shared__ __attribute__((aligned(16))) Turned<float, NT> ut;            // dU on its way out
  __shared__ __attribute__((aligned(16))) Gates gate[4];                   // by the chunk's number modulo 4

  int64_t unit;
  int part;
  if (!gdr_block(blockIdx.x, p.n_seq * p.Hv, p.dv / (16 * NT), &unit, &part)) return;
  const int64_t s = unit / p.Hv;
  const int h = (int)(unit % p.Hv), kh = h / (p.Hv / p.Hk);
  const GdrSeq seq = gdr_seq(p, s);
  const int64_t nc = seq.n_chunks;
  const int lane = threadIdx.x & 63, li = lane & 15, g = lane >> 4;
  const int wave = wave_id() & 3;
  const int col0 = 16 * NT * part;
  const int r0 = 16 * wave + 4 * g;
  const int last_rows = (int)(seq.len - (nc - 1) * kGdrChunk);
  const bool owner = wave * RT < DK / 16;
  const int first_tile = owner ? wave * RT : 0;
  const int64_t blk0 = seq.slot0 * p.Hv + h;
  const auto gates = global_in<float>(p.ws_gate) + blk0 * kGateFloats;

  if (wave_id() < 4) {
    floatx4 S[NT][RT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int m = 0; m < RT; ++m) {
        S[nt][m] = floatx4{};
        if (owner && p.dSf) {
          const auto at = global_in<float>(p.dSf) + unit * p.dk * p.dv + (16 * (wave * RT + m) + 4 * g) * p.dv + col0 + 16 * nt + li;
#pragma unroll
          for (int r = 0; r < 4; ++r) S[nt][m][r] = at[r * p.dv];
        }
      }
    auto put_state = [&]() {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int m = 0; m < RT; ++m) {
          const int t = wave * RT + m;
          if (owner) put_op<3>(sf[nt] + (t >> 1) * kOp3, t & 1, li, g, S[nt][m], T{});
        }
    };
    put_state();
    auto walk = [&](auto both) {
      constexpr int TS = decltype(both)::value ? 2 : 1;   // T^T of wavefronts 0 and 1 reaches into both steps
      struct Buf {
        In k[KS];
        Op3 tt[TS];
      };
      // where the next loads come from: the last chunk, then downwards
      int64_t at = nc - 1;
      auto kp = global_in<T>(p.k) + seq.row * p.sk.b + kh * p.sk.h + (seq.t0 + at * kGdrChunk) * p.sk.t;
      auto tp = as_global((const char*)p.ws_tt) + (blk0 + at * p.Hv) * kTriFrags * kOp3 + upper_frag(wave, wave < 2 ? 0 : 1) * kOp3;
      const LaneRow krow(16 * wave + li, last_rows, p.sk.t, 8 * g, sizeof(T));
      auto load_k = [&](Buf& b) {
        const auto from = lane_at(kp, krow.of(at == nc - 1));
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) b.k[ks] = load_row8(from + 32 * ks);
      };
      auto load_tt = [&](Buf& b) {
#pragma unroll
        for (int ks = 0; ks < TS; ++ks) b.tt[ks] = load_frag<Op3>(tp + ks * kOp3, lane);
        const int64_t more = mask_of(at > 0);
        at -= more & 1;
        kp -= more & (int64_t)(kGdrChunk * p.sk.t);
        tp -= more & (int64_t)(p.Hv * (kTriFrags * kOp3));
      };
      auto step = [&](Buf& b, int64_t c, int n) {
        const Gates& gt = gate[c & 3];
        const floatx4 eta = ld4f((const float*)gt.eta + r0);
        floatx4 X[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          Op3 sb[KS];
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) sb[ks] = load_frag<Op3>((const char*)sf[nt] + ks * kOp3, lane);
          X[nt] = mma_steps(b.k, sb, floatx4{});
        }
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) kl.put8(16 * wave + li, 32 * ks + 8 * g, b.k[ks]);
        load_k(b);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const floatx4 first = ld4f((const float*)&x0[nt][(wave * 64 + lane) * 4]);
#pragma unroll
          for (int r = 0; r < 4; ++r) X[nt][r] = r0 + r < n ? eta[r] * X[nt][r] + first[r] : 0.f;
          put_op<3>(xf[nt] + (wave >> 1) * kOp3, wave & 1, li, g, X[nt], T{});
        }
        block_barrier();

        const floatx4 gam = ld4f((const float*)gt.gam + r0), beta = ld4f((const float*)gt.beta + r0);
        floatx4 dU[NT], add[NT][RT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          Op3 xb[TS];
#pragma unroll
          for (int ks = 0; ks < TS; ++ks) xb[ks] = load_frag<Op3>((const char*)xf[nt] + (ks + 2 - TS) * kOp3, lane);
#pragma unroll
          for (int m = 0; m < RT; ++m) add[nt][m] = ld4f((const float*)&d0[nt][((first_tile + m) * 64 + lane) * 4]);
          dU[nt] = mma_steps(b.tt, xb, floatx4{});
        }
        load_tt(b);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          put_op<3>(ef[nt] + (wave >> 1) * kOp3, wave & 1, li, g, -(gam * beta) * dU[nt], T{});
          ut.put_tile(16 * nt + li, r0, dU[nt]);
        }
        block_barrier();

        In kt[RT][2];
#pragma unroll
        for (int m = 0; m < RT; ++m)
#pragma unroll
          for (int ks = 0; ks < 2; ++ks) kt[m][ks] = kl.transposed(first_tile + m, ks, lane);
        const float last = gt.gam[63];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const Op3 eb[2] = {load_frag<Op3>((const char*)ef[nt], lane), load_frag<Op3>((const char*)ef[nt] + kOp3, lane)};
#pragma unroll
          for (int m = 0; m < RT; ++m) S[nt][m] = mma_steps(kt[m], eb, S[nt][m] * last + add[nt][m]);
        }
        put_state();
        block_barrier();
      };
      if (nc > 0) {
        Buf buf[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          load_k(buf[i]);
          load_tt(buf[i]);
        }
        int64_t c = nc - 1;
        step(buf[0], c--, last_rows);
        if (kAhead == 1) {
          for (; c >= 0; --c) step(buf[0], c, kGdrChunk);
        } else {
          for (; c > 0; c -= 2) {
            step(buf[kAhead - 1], c, kGdrChunk);
            step(buf[0], c - 1, kGdrChunk);
          }
          if (c == 0) step(buf[kAhead - 1], c, kGdrChunk);
        }
      }
    };
    block_barrier();
    block_barrier();
    block_barrier();
    if (wave < 2) walk(std::true_type{});
    else walk(std::false_type{});
    if (p.dS0 && owner) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int m = 0; m < RT; ++m) {
          const auto at = global_out<float>(p.dS0) + unit * p.dk * p.dv + (16 * (wave * RT + m) + 4 * g) * p.dv + col0 + 16 * nt + li;
#pragma unroll
          for (int r = 0; r < 4; ++r) at[r * p.dv] = S[nt][m][r];
        }
    }
    return;
  }

  // wavefronts 4-7: dO and the gates are fetched two chunks ahead of the chain and turned in LDS, what they make
  // is ready one chunk ahead
  auto serve = [&](auto both) {
    constexpr int TS = decltype(both)::value ? 2 : 1;
    const int tid = threadIdx.x & 255;
    In ox, fx;
    float gx = 0.f;
    Op3 pm[TS];
    In q[KS];
    int64_t at = nc - 1, pat = nc - 1;   // the chunk that is fetched next, and whose P and Q are loaded next
    auto dop = global_in<T>(p.dO) + seq.row * p.sdo.b + h * p.sdo.h + (seq.t0 + at * kGdrChunk) * p.sdo.t + col0;
    auto gp = gates + at * p.Hv * kGateFloats + (wave < 3 ? wave : 0) * 64;
    auto pp = as_global((const char*)p.ws_p) + ((blk0 + at * p.Hv) * kTriFrags + upper_frag(wave, TS == 2 ? 0 : 1)) * kOp3;
    auto qp = global_in<T>(p.q) + seq.row * p.sq.b + kh * p.sq.h + (seq.t0 + at * kGdrChunk) * p.sq.t;
    // of the chunk the chain is at
    auto fp = global_in<T>(p.ws_f) + (blk0 + at * p.Hv) * kGdrChunk * p.dv + col0;
    auto sp = global_out<T>(p.ws_ds) + (blk0 + at * p.Hv) * p.dk * p.dv + col0;
    auto dvp = global_out<T>(p.dv_) + seq.row * p.sdv.b + h * p.sdv.h + (seq.t0 + at * kGdrChunk) * p.sdv.t + col0;
    auto dbp = global_out<float>(p.ws_db) + ((blk0 + at * p.Hv) * (p.dv / (16 * NT)) + part) * kGdrChunk;
    const int row = tid / kPer;          // this thread's token of dO, F and dU
    const LaneRow orow(row, last_rows, p.sdo.t, 8 * (tid % kPer), sizeof(T));
    const LaneRow qrow(16 * wave + li, last_rows, p.sq.t, 8 * g, sizeof(T));
    const uint32_t frow = (uint32_t)((row * p.dv + 8 * (tid % kPer)) * sizeof(T));
    const uint32_t vrow = (uint32_t)((row * p.sdv.t + 8 * (tid % kPer)) * sizeof(T));
    auto fetch = [&]() {
      if (wave < kPer) ox = load_row8(lane_at(dop, orow.of(at == nc - 1)));
      if (wave < 3) gx = *lane_at(gp, lane * 4);
      const int64_t more = mask_of(at > 0);
      at -= more & 1;
      dop -= more & (int64_t)(kGdrChunk * p.sdo.t);
      gp -= more & (int64_t)(p.Hv * kGateFloats);
    };
    auto leave = [&](int64_t c) {
      if (wave < kPer) ot.put_row(tid, ox);
      if (wave < 3) (wave == 0 ? gate[c & 3].gam : wave == 1 ? gate[c & 3].eta : gate[c & 3].beta)[lane] = gx;
    };
    auto load_pq = [&]() {
#pragma unroll
      for (int ks = 0; ks < TS; ++ks) pm[ks] = load_frag<Op3>(pp + ks * kOp3, lane);
      const auto from = lane_at(qp, qrow.of(pat == nc - 1));
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) q[ks] = load_row8(from + 32 * ks);
      const int64_t more = mask_of(pat > 0);
      pat -= more & 1;
      pp -= more & (int64_t)(p.Hv * (kTriFrags * kOp3));
      qp -= more & (int64_t)(kGdrChunk * p.sq.t);
    };
    auto load_f = [&](int64_t c) {
      if (wave < kPer) fx = load_row8(lane_at(fp, frow));
      fp -= mask_of(c > 0) & (int64_t)(p.Hv * (kGdrChunk * p.dv));
    };
    auto spread = [&](int64_t c) {       // dO of chunk c as operands, and its Q
      const int n = c == nc - 1 ? last_rows : kGdrChunk;
      const floatx4 gam = p.scale * ld4f((const float*)gate[c & 3].gam + r0);
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) ql.put8(16 * wave + li, 32 * ks + 8 * g, q[ks]);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        floatx4 x = ot.tile(16 * nt + li, r0);
#pragma unroll
        for (int r = 0; r < 4; ++r) x[r] = r0 + r < n ? x[r] : 0.f;
        put_op<1>(of[nt] + (wave >> 1) * kIn, wave & 1, li, g, x, T{});
        put_op<3>(gf[nt] + (wave >> 1) * kOp3, wave & 1, li, g, gam * x, T{});
      }
    };
    // x0 and d0 are read by the chain before this chunk's second barrier and written after it
    floatx4 X[NT], D[NT][RT];
    auto products = [&]() {
      In qt[RT][2];
#pragma unroll
      for (int m = 0; m < RT; ++m)
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) qt[m][ks] = ql.transposed(first_tile + m, ks, lane);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        X[nt] = mma(pm[TS - 1], load_frag<In>((const char*)of[nt] + kIn, lane), floatx4{});
        if constexpr (TS == 2) X[nt] = mma(pm[0], load_frag<In>((const char*)of[nt], lane), X[nt]);
        const Op3 gb[2] = {load_frag<Op3>((const char*)gf[nt], lane), load_frag<Op3>((const char*)gf[nt] + kOp3, lane)};
#pragma unroll
        for (int m = 0; m < RT; ++m) D[nt][m] = mma_steps(qt[m], gb, floatx4{});
      }
      load_pq();
    };
    auto leave_products = [&]() {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        *reinterpret_cast<floatx4*>(&x0[nt][(wave * 64 + lane) * 4]) = X[nt];
#pragma unroll
        for (int m = 0; m < RT; ++m)
          if (owner) *reinterpret_cast<floatx4*>(&d0[nt][((wave * RT + m) * 64 + lane) * 4]) = D[nt][m];
      }
    };
    // dU as the chain has left it: the gradient of v, and beta's over these columns
    auto finish = [&](int64_t c) {
      const int n = c == nc - 1 ? last_rows : kGdrChunk;
      if (wave < kPer) {
        const float b = gate[c & 3].beta[row];
        const float8v dU = ut.row(tid);
        T f8[8];
        __builtin_memcpy(f8, &fx, sizeof(fx));
        float x = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) x += dU[e] * value(f8[e]);
#pragma unroll
        for (int d = 1; d < kPer; d <<= 1) x += __shfl_xor(x, d);
        if (tid % kPer == 0) *lane_at(dbp, row * 4) = x;
        if (row < n) {
          store_row4(lane_at(dvp, vrow), b * floatx4{dU[0], dU[1], dU[2], dU[3]});
          store_row4(lane_at(dvp, vrow + 4 * sizeof(T)), b * floatx4{dU[4], dU[5], dU[6], dU[7]});
        }
      }
      dvp -= kGdrChunk * p.sdv.t;
      dbp -= p.Hv * (p.dv / (16 * NT) * kGdrChunk);
    };
    if (nc > 0) {
      fetch();
      load_pq();
      load_f(nc - 1);
      leave(nc - 1);
      fetch();
    }
    block_barrier();
    if (nc > 0) spread(nc - 1);
    block_barrier();
    if (nc > 0) {
      products();
      leave_products();
      leave(nc - 2);
      fetch();
    }
    block_barrier();
    for (int64_t c = nc - 1; c >= 0; --c) {
      // dS at this chunk's end; what the chain needs of the next one
      write_rows<T, NT>(sf[0], kOp3, KS * kOp3, DK, sp, p.dv, tid);
      sp -= p.Hv * (p.dk * p.dv);
      if (c > 0) spread(c - 1);
      block_barrier();
      if (c > 0) products();
      block_barrier();
      if (c > 0) leave_products();
      finish(c);
      load_f(c - 1);
      leave(c - 2);
      fetch();
      block_barrier();
    }
  };
  if (wave < 2) serve(std::true_type{});
  else serve(std::false_type{});
}

template <typename T, int DK, int NT>
hipError_t launch_scan(const GdrParams& p, hipStream_t s, int kind) {
  const dim3 grid((unsigned)gdr_blocks(p.n_seq * p.Hv, p.dv / (16 * NT)));
  if (kind == 0) hipLaunchKernelGGL((gdr_scan_kernel<T, DK, NT, false>), grid, dim3(512), 0, s, p);
  else if (kind == 1) hipLaunchKernelGGL((gdr_scan_kernel<T, DK, NT, true>), grid, dim3(512), 0, s, p);
  else hipLaunchKernelGGL((gdr_rscan_kernel<T, DK, NT>), grid, dim3(512), 0, s, p);
  return hipGetLastError();
}

template <typename T>
hipError_t launch_t(const GdrParams& p, hipStream_t s, int kind) {
  constexpr int NT = sizeof(T) == 2 ? kGdrTilesBf16 : 1;
  switch (p.dk) {
    case 32: return launch_scan<T, 32, NT>(p, s, kind);
    case 64: return launch_scan<T, 64, NT>(p, s, kind);
    default: return launch_scan<T, 128, NT>(p, s, kind);
  }
}

hipError_t launch_kind(const GdrParams& p, hipStream_t s, int kind) {
  return p.dtype == KDA_DTYPE_BF16 ? launch_t<uint16_t>(p, s, kind) : launch_t<float>(p, s, kind);
}

}  // namespace

hipError_t launch_gdr_scan(const GdrParams& p, hipStream_t s, bool states) { return launch_kind(p, s, states ? 1 : 0); }
hipError_t launch_gdr_rscan(const GdrParams& p, hipStream_t s) { return launch_kind(p, s, 2); }

}  // namespace kda
