// The sequential part of the head-gated delta rule: the state from chunk to chunk, and the outputs.
//
// Value columns are independent, so a workgroup owns one (sequence, value head) and 16 of its columns and
// walks the chunks:
//   E = V - gam K S  |  U = beta T' E  |  S <- e^{G_last} S + K^T (eta U)         O = scale gam Q S + P U
// with a barrier at each bar.  What bounds it is that chain: three products of 16 columns, each waiting
// for the one before, so everything else is kept off it.
//  - Wavefronts 0-3 walk the chain.  Wavefront i owns token rows 16i .. 16i + 15 and a quarter of the
//    state's rows, in registers (fp32 matrix-core results).  Wavefronts 4-7, one more on each SIMD, form the
//    outputs (or, in the backward's run, write out the entering states and F) in the chain's shadow, and move
//    v, o and the gates in rows of 16 bytes a lane, turning them in LDS.
//  - A step's bytes matter too (62 KiB, 19 a cycle for a compute unit): K is loaded once, as whole rows, and LDS
//    gives both its row and its transposed operands; loads are spread over the three parts of a step and issued as
//    soon as the registers they go to are free, one step ahead.  Loads past the last chunk are clamped to it.
//  - What the wavefronts exchange (the state, E, U: 16 columns each) goes through LDS as ready B operands.
// 64K tokens of 16 heads (dk = dv = 128, bf16): 1.42 ms, 3250 cycles for a step of 64 tokens, of which the chain's
// wavefronts work 2500 to 2900 and wait for the serving ones or for each other the rest.  32 columns a workgroup:
// 4400 cycles, with half the workgroups; two workgroups a compute unit (128 registers) spill and take 2.8 ms.
// Rows behind the sequence's end read its last row; their E is set to zero, so nothing of them reaches
// the state, and their outputs are not written.
#include <type_traits>

#include "gdr_internal.h"

namespace kda {

namespace {

constexpr int kScanWaves = 2;   // wavefronts a SIMD that the registers are to allow

__device__ __forceinline__ float value(uint16_t x) { return bf16_to_f32(x); }
__device__ __forceinline__ float value(float x) { return x; }

// Writes `rows` contraction places x 16 columns of B operands to memory, place by place, bf16 in two planes of `plane`
// values: a lane takes 8 columns of one place.  A workgroup's 16 columns lie together there (as 32 bytes of rows of
// all columns, 2x4096 tokens' two chains took 126 and 220 us in place of 109 and 201).  bf16: transposing reads, in which 16 lanes read 16 places
// of 4 columns and get one place's 4 columns each.
template <typename T>
__device__ __forceinline__ void write_rows(const char* frags, int frag_bytes, int rows, GlobalPtr<T> out, int64_t plane, int tid) {
  if constexpr (sizeof(T) == 2) {
    typedef __attribute__((address_space(3))) bf16x4 lds_bf16x4;
    const int group = tid >> 4, j = tid & 15, block = group >> 1, c0 = (group & 1) * 8;   // block of 16 places
    if (16 * block >= rows) return;   // whole wavefronts: rows are a multiple of 32
    const char* fr = frags + (block >> 1) * frag_bytes + (c0 + (j >> 2) + 16 * (2 * (block & 1) + ((j >> 1) & 1))) * 16 + (j & 1) * 8;
#pragma unroll
    for (int n = 0; n < kKept<T>; ++n) {
      const bf16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_bf16x4*)(fr + n * kPlane));
      const bf16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_bf16x4*)(fr + n * kPlane + 4 * 16));
      *repoint<bf16x8>(out + n * plane + (16 * block + j) * 16 + c0) =
          __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    }
  } else {
    for (int i = tid; i < rows * 2; i += 256) {
      const int r = i >> 1, c0 = (i & 1) * 8;
      float8v x;
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = frag_at<T>(frags + (r >> 5) * frag_bytes, r & 31, c0 + e);
      *repoint<float8v>(out + r * 16 + c0) = x;
    }
  }
}

// All ones or zeros, of a condition on values of the wavefront.  Positions advance by masked amounts, not
// behind a branch, which would come between matrix instructions and the reads of their results (see settle).
__device__ __forceinline__ int64_t mask_of(bool c) { return __builtin_amdgcn_readfirstlane(c ? -1 : 0); }

// Byte offset, from a chunk's first row, of what a lane reads of row `row` of a strided tensor; in the last
// chunk the rows behind the sequence's end become its last one.
struct LaneRow {
  uint32_t whole, tail;
  __device__ __forceinline__ LaneRow(int row, int last_rows, int64_t stride, int at, int esz)
      : whole((uint32_t)((row * stride + at) * esz)), tail((uint32_t)((min(row, last_rows - 1) * stride + at) * esz)) {}
  LaneRow() = default;
  __device__ __forceinline__ uint32_t of(bool last) const { return last ? tail : whole; }
};

// A wavefront's 16 rows of K or Q, whole rows at a time, and where the next chunk's are
template <typename T, int DK> struct RowLoads {
  static constexpr int kLoads = DK / 32, kPieces = DK / 8;
  typename Frags<T>::In v[kLoads];
  LaneRow at[kLoads];
  GlobalPtr<const T> from;
  __device__ __forceinline__ RowLoads(GlobalPtr<const T> first, int wave, int lane, int last_rows, int64_t stride) : from(first) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
      at[i] = LaneRow(16 * wave + (64 * i + lane) / kPieces, last_rows, stride, (64 * i + lane) % kPieces * 8, sizeof(T));
  }
  __device__ __forceinline__ void load(bool last) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) v[i] = load_row8(lane_at(from, at[i].of(last)));
  }
};

// 64 tokens x 16 columns in LDS, column by column (a result tile's lane reads 4 tokens of its column).
// Threads 0 .. 127 of four wavefronts move them: thread t has columns 8 (t & 1) .. + 7 of token t / 2.
template <typename T> struct Turned {
  static constexpr int kLd = sizeof(T) == 2 ? 72 : 68;
  T x[16 * kLd];
  __device__ __forceinline__ void put_row(int t, const typename Frags<T>::In& v) {
    T e8[8];
    __builtin_memcpy(e8, &v, sizeof(v));
#pragma unroll
    for (int e = 0; e < 8; ++e) x[(8 * (t & 1) + e) * kLd + (t >> 1)] = e8[e];
  }
  __device__ __forceinline__ typename Frags<T>::In row(int t) const {
    T e8[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) e8[e] = x[(8 * (t & 1) + e) * kLd + (t >> 1)];
    typename Frags<T>::In v;
    __builtin_memcpy(&v, e8, sizeof(v));
    return v;
  }
  __device__ __forceinline__ floatx4 tile(int li, int r0) const {
    if constexpr (sizeof(T) == 2) {
      const u32x2v p = *reinterpret_cast<const u32x2v*>(x + li * kLd + r0);
      return floatx4{lo_bf16(p[0]), hi_bf16(p[0]), lo_bf16(p[1]), hi_bf16(p[1])};
    } else {
      return *reinterpret_cast<const floatx4*>(x + li * kLd + r0);
    }
  }
  __device__ __forceinline__ void put_tile(int li, int r0, floatx4 v) {
    if constexpr (sizeof(T) == 2) *reinterpret_cast<u32x2v*>(x + li * kLd + r0) = u32x2v{pk_bf16(v[0], v[1]), pk_bf16(v[2], v[3])};
    else *reinterpret_cast<floatx4*>(x + li * kLd + r0) = v;
  }
};
// The sequence that the i-th workgroups of a packed batch take: the i-th longest, as far as a thread each can find
// the order.  One workgroup fills a compute unit, and a long sequence that starts last would run alone at the end
// (prompts of 517, 0, 1, 64, 1300, 63, 65, 2000 and 89 tokens of 16 heads: 79 us in their order, 71 so).
__device__ __forceinline__ int64_t by_length(const GdrParams& p, int64_t i) {
  constexpr int kMost = 512;   // threads of a workgroup
  __shared__ int chunks[kMost], found;
  if (!p.seq_start || p.n_seq < 2 || p.n_seq > kMost) return i;
  const int me = threadIdx.x, n = (int)p.n_seq;
  const int mine = me < n ? (int)gdr_seq(p, me).n_chunks : 0;
  chunks[me] = mine;
  __syncthreads();
  int before = 0;
  for (int j = 0; j < n; ++j) before += chunks[j] > mine || (chunks[j] == mine && j < me);
  if (me < n && before == (int)i) found = me;
  __syncthreads();
  return __builtin_amdgcn_readfirstlane(found);
}

// a chunk's gates in LDS
struct Gates {
  float gam[64], eta[64], beta[64];
};
static_assert(kGateGam == 0 && kGateEta == 64 && kGateBeta == 128, "a wavefront each");

template <typename T, int DK, bool STATES>
__global__ __launch_bounds__(512, kScanWaves) void gdr_scan_kernel(GdrParams p) {
  using In = typename Frags<T>::In;
  using Op3 = typename Frags<T>::template Op<3>;
  using Op2 = typename Frags<T>::template Op<2>;
  constexpr int KS = DK / 32;
  constexpr int RT = DK >= 64 ? DK / 64 : 1;      // state row tiles of a wavefront
  constexpr int kOp2 = op_frag<T, 2>(), kOp3 = op_frag<T, 3>();
  __shared__ __attribute__((aligned(16))) char sf[KS * kOp3];              // the state, as B operands
  __shared__ __attribute__((aligned(16))) char ef[2 * kOp3];               // E
  __shared__ __attribute__((aligned(16))) char wf[2 * kOp3];               // eta U
  __shared__ __attribute__((aligned(16))) char uf[2 * kOp2];               // U (F where states are written)
  __shared__ __attribute__((aligned(16))) Rows<T, DK> kl;                  // the chunk's K
  __shared__ __attribute__((aligned(16))) Rows<T, STATES ? 32 : DK> ql;    // and Q
  __shared__ __attribute__((aligned(16))) Turned<T> vt[2];                 // v, by the chunk's parity
  __shared__ __attribute__((aligned(16))) Turned<T> ot;                    // o on its way out
  __shared__ __attribute__((aligned(16))) Gates gate[2];

  int64_t unit;
  int part;
  if (!gdr_block(blockIdx.x, p.n_seq * p.Hv, p.dv / 16, &unit, &part)) return;
  const int h = (int)(unit % p.Hv), kh = h / (p.Hv / p.Hk);
  const int64_t s = by_length(p, unit / p.Hv);
  unit = s * p.Hv + h;
  const GdrSeq seq = gdr_seq(p, s);
  const int64_t nc = seq.n_chunks;
  const int lane = threadIdx.x & 63, li = lane & 15, g = lane >> 4;
  const int wave = wave_id() & 3;
  const int col = 16 * part + li;
  const int r0 = 16 * wave + 4 * g;               // first of this lane's 4 token rows in result tiles
  const int last_rows = (int)(seq.len - (nc - 1) * kGdrChunk);   // tokens of the last chunk
  const int64_t blk0 = seq.slot0 * p.Hv + h;      // workspace block of chunk 0; the next is Hv further

  if (wave_id() < 4) {
    const bool owner = wave * RT < DK / 16;
    const int first_tile = owner ? wave * RT : 0;
    floatx4 S[RT];
#pragma unroll
    for (int m = 0; m < RT; ++m) {
      S[m] = floatx4{};
      if (owner && p.S0) {
        const auto at = global_in<float>(p.S0) + unit * p.dk * p.dv + (16 * (wave * RT + m) + 4 * g) * p.dv + col;
#pragma unroll
        for (int r = 0; r < 4; ++r) S[m][r] = at[r * p.dv];
      }
    }
    auto put_state = [&]() {
#pragma unroll
      for (int m = 0; m < RT; ++m) {
        const int t = wave * RT + m;
        if (owner) put_op<3>(sf + (t >> 1) * kOp3, t & 1, li, g, S[m], T{});
      }
    };
    put_state();

    // BOTH: the wavefront's rows of T' reach into both steps of 32 tokens (wavefronts 2 and 3)
    auto walk = [&](auto both) {
      constexpr int TS = decltype(both)::value ? 2 : 1;
      RowLoads<T, DK> kr(global_in<T>(p.k) + seq.row * p.sk.b + kh * p.sk.h + seq.t0 * p.sk.t, wave, lane, last_rows, p.sk.t);
      auto tp = as_global((const char*)p.ws_ti) + blk0 * kTriFrags * kOp3 + lower_frag(wave, 0) * kOp3;
      int64_t k_at = 0, t_at = 0;    // the chunks whose K and T' are loaded next
      In kf[KS];
      Op3 ti[TS];
      auto load_k = [&]() {
        kr.load(k_at == nc - 1);
        const int64_t more = mask_of(k_at < nc - 1);
        k_at += more & 1;
        kr.from += more & (int64_t)(kGdrChunk * p.sk.t);
      };
      auto turn_k = [&]() {          // the loaded K to LDS, and this wavefront's rows back
        kl.leave(kr.v, 16 * wave, lane);
        load_k();
        compiler_fence();
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) kf[ks] = kl.row_frag(wave, ks, lane);
      };
      auto load_ti = [&]() {
#pragma unroll
        for (int ks = 0; ks < TS; ++ks) ti[ks] = load_frag<Op3>(tp + ks * kOp3, lane);
        const int64_t more = mask_of(t_at < nc - 1);
        t_at += more & 1;
        tp += more & (int64_t)(p.Hv * (kTriFrags * kOp3));
      };
      auto step = [&](int64_t c, int n) {
        const Gates& gt = gate[c & 1];
        Op3 sb[KS];
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) sb[ks] = load_frag<Op3>((const char*)sf + ks * kOp3, lane);
        const floatx4 v = vt[c & 1].tile(li, r0), gam = ld4f((const float*)gt.gam + r0);
        floatx4 E = mma_steps(kf, sb, floatx4{});
#pragma unroll
        for (int r = 0; r < 4; ++r) E[r] = r0 + r < n ? v[r] - gam[r] * E[r] : 0.f;
        put_op<3>(ef + (wave >> 1) * kOp3, wave & 1, li, g, E, T{});
        block_barrier();

        Op3 eb[TS];
#pragma unroll
        for (int ks = 0; ks < TS; ++ks) eb[ks] = load_frag<Op3>((const char*)ef + ks * kOp3, lane);
        const floatx4 eta = ld4f((const float*)gt.eta + r0), beta = ld4f((const float*)gt.beta + r0);
        const float last = gt.gam[63];   // e^{G_last}: tokens behind the end do not decay
        In kt[RT][2];
#pragma unroll
        for (int m = 0; m < RT; ++m)
#pragma unroll
          for (int ks = 0; ks < 2; ++ks) kt[m][ks] = kl.transposed(first_tile + m, ks, lane);
        const floatx4 F = mma_steps(ti, eb, floatx4{});
        load_ti();
        const floatx4 U = beta * F;
        put_op<3>(wf + (wave >> 1) * kOp3, wave & 1, li, g, eta * U, T{});
        block_barrier();

        const Op3 wb[2] = {load_frag<Op3>((const char*)wf, lane), load_frag<Op3>((const char*)wf + kOp3, lane)};
        put_op<2>(uf + (wave >> 1) * kOp2, wave & 1, li, g, STATES ? F : U, T{});
#pragma unroll
        for (int m = 0; m < RT; ++m) S[m] = mma_steps(kt[m], wb, S[m] * last);
        turn_k();
        put_state();
        block_barrier();
      };
      if (nc > 0) {
        load_k();
        load_ti();
        turn_k();
      }
      block_barrier();
      for (int64_t c = 0; c < nc; ++c) step(c, c == nc - 1 ? last_rows : kGdrChunk);
    };
    if (wave < 2) walk(std::false_type{});
    else walk(std::true_type{});
    if constexpr (!STATES) block_barrier();   // the last chunk's outputs, between wavefronts 4-7
    if (p.S_final && owner) {
#pragma unroll
      for (int m = 0; m < RT; ++m) {
        const auto at = global_out<float>(p.S_final) + unit * p.dk * p.dv + (16 * (wave * RT + m) + 4 * g) * p.dv + col;
#pragma unroll
        for (int r = 0; r < 4; ++r) at[r * p.dv] = S[m][r];
      }
    }
    return;
  }

  // v and the gates of one chunk ahead of the chain: loaded, then left in LDS
  const int tid = threadIdx.x & 255;
  In vx;
  float gx = 0.f;
  int64_t ahead = 0;
  auto vp = global_in<T>(p.v) + seq.row * p.sv.b + h * p.sv.h + seq.t0 * p.sv.t + 16 * part;
  auto gp = global_in<float>(p.ws_gate) + blk0 * kGateFloats + (wave < 3 ? wave : 0) * 64;
  const LaneRow vrow(tid >> 1, last_rows, p.sv.t, 8 * (tid & 1), sizeof(T));
  auto fetch = [&]() {
    if (wave < 2) vx = load_row8(lane_at(vp, vrow.of(ahead == nc - 1)));
    if (wave < 3) gx = *lane_at(gp, lane * 4);
    const int64_t more = mask_of(ahead < nc - 1);
    ahead += more & 1;
    vp += more & (int64_t)(kGdrChunk * p.sv.t);
    gp += more & (int64_t)(p.Hv * kGateFloats);
  };
  auto leave = [&](int64_t c) {
    if (wave < 2) vt[c & 1].put_row(tid, vx);
    if (wave < 3) (wave == 0 ? gate[c & 1].gam : wave == 1 ? gate[c & 1].eta : gate[c & 1].beta)[lane] = gx;
  };
  if (nc > 0) {
    fetch();
    leave(0);
    fetch();
  }
  if constexpr (STATES) {
    block_barrier();   // the first state, v and gates
    const int64_t s_plane = p.dk * p.dv, f_plane = kGdrChunk * p.dv;
    auto sp = global_out<T>(p.ws_s) + blk0 * kKept<T> * s_plane + part * (DK * 16);
    auto fp = global_out<T>(p.ws_f) + blk0 * kKept<T> * f_plane + part * (kGdrChunk * 16);
    for (int64_t c = 0; c < nc; ++c) {
      // F of the chunk before; the state that enters this one; what the chain needs of the next
      if (c > 0) {
        write_rows<T>(uf, kOp2, kGdrChunk, fp, f_plane, tid);
        fp += p.Hv * kKept<T> * f_plane;
      }
      block_barrier();
      write_rows<T>(sf, kOp3, DK, sp, s_plane, tid);
      sp += p.Hv * kKept<T> * s_plane;
      block_barrier();
      leave(c + 1);
      fetch();
      block_barrier();
    }
    if (nc > 0) write_rows<T>(uf, kOp2, kGdrChunk, fp, f_plane, tid);
  } else {
    auto op = global_out<T>(p.o) + seq.row * p.so.b + h * p.so.h + seq.t0 * p.so.t + 16 * part;
    const uint32_t orow = (uint32_t)(((tid >> 1) * p.so.t + 8 * (tid & 1)) * sizeof(T));
    auto store = [&](int n) {
      if (tid < 2 * n) *repoint<In>(lane_at(op, orow)) = ot.row(tid);
      op += kGdrChunk * p.so.t;
    };
    auto walk = [&](auto both) {
      constexpr int TS = decltype(both)::value ? 2 : 1;
      RowLoads<T, DK> qr(global_in<T>(p.q) + seq.row * p.sq.b + kh * p.sq.h + seq.t0 * p.sq.t, wave, lane, last_rows, p.sq.t);
      auto pp = as_global((const char*)p.ws_p) + blk0 * kTriFrags * kOp2 + lower_frag(wave, 0) * kOp2;
      int64_t q_at = 0, p_at = 0;
      In qf[KS];
      Op2 pm[TS];
      auto load_q = [&]() {
        qr.load(q_at == nc - 1);
        const int64_t more = mask_of(q_at < nc - 1);
        q_at += more & 1;
        qr.from += more & (int64_t)(kGdrChunk * p.sq.t);
      };
      auto turn_q = [&]() {          // through this wavefront's own rows of LDS
        ql.leave(qr.v, 16 * wave, lane);
        load_q();
        compiler_fence();
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) qf[ks] = ql.row_frag(wave, ks, lane);
      };
      auto load_p = [&]() {
#pragma unroll
        for (int ks = 0; ks < TS; ++ks) pm[ks] = load_frag<Op2>(pp + ks * kOp2, lane);
        const int64_t more = mask_of(p_at < nc - 1);
        p_at += more & 1;
        pp += more & (int64_t)(p.Hv * (kTriFrags * kOp2));
      };
      floatx4 O = {};
      // the outputs of a chunk whose U the chain has left; two planes of P, U and the state, as o is rounded to
      // the inputs' type
      auto add_own = [&]() {
        Op2 ub[TS];
#pragma unroll
        for (int ks = 0; ks < TS; ++ks) ub[ks] = load_frag<Op2>((const char*)uf + ks * kOp2, lane);
        O = mma_steps(pm, ub, O);
        load_p();
        settle(O);
        ot.put_tile(li, r0, O);
      };
      if (nc > 0) {
        load_q();
        load_p();
        turn_q();
      }
      block_barrier();   // the first state, v and gates
      for (int64_t c = 0; c < nc; ++c) {
        if (c > 0) add_own();                   // finishes the chunk before
        block_barrier();
        Op2 sb[KS];
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) sb[ks] = load_frag<Op2>((const char*)sf + ks * kOp3, lane);
        const floatx4 gam = ld4f((const float*)gate[c & 1].gam + r0);
        O = mma_steps(qf, sb, floatx4{});
        settle(O);
        O = (p.scale * gam) * O;
        block_barrier();
        if (c > 0) store(kGdrChunk);
        turn_q();
        leave(c + 1);
        fetch();
        block_barrier();
      }
      if (nc > 0) add_own();
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
// chain leaves, per 16 columns, the sums of dU F that make beta's gradient.  2 x 4096 tokens of 16 heads: 204 us.
// The serving wavefronts set the pace: of a step's 5900 cycles they work about 5000, wavefronts 0-3 about 2900.
// (At 192 us, a copy without P^T's loads and products took 158; formed by the preparation kernel instead, P^T dO cost
// that kernel 23 us more and saved 17 here.)
template <typename T, int DK>
__global__ __launch_bounds__(512, kScanWaves) void gdr_rscan_kernel(GdrParams p) {
  using In = typename Frags<T>::In;
  using Op3 = typename Frags<T>::template Op<3>;
  constexpr int KS = DK / 32;
  constexpr int RT = DK >= 64 ? DK / 64 : 1;
  constexpr int kIn = in_frag<T>(), kOp3 = op_frag<T, 3>();
  __shared__ __attribute__((aligned(16))) char sf[KS * kOp3];          // dS
  __shared__ __attribute__((aligned(16))) char xf[2 * kOp3];           // X
  __shared__ __attribute__((aligned(16))) char ef[2 * kOp3];           // -gam dE
  __shared__ __attribute__((aligned(16))) char of[2 * kIn];            // dO
  __shared__ __attribute__((aligned(16))) char gf[2 * kOp3];           // scale gam dO
  __shared__ __attribute__((aligned(16))) float x0[4 * 256];           // P^T dO, result tiles [wave][lane][4]
  __shared__ __attribute__((aligned(16))) float d0[DK / 16 * 256];     // Q^T (scale gam dO)
  __shared__ __attribute__((aligned(16))) Rows<T, DK> kl, ql;              // the chain's K, the next chunk's Q
  __shared__ __attribute__((aligned(16))) Turned<T> ot;                // dO on its way in
  __shared__ __attribute__((aligned(16))) Turned<float> ut;            // dU on its way out
  __shared__ __attribute__((aligned(16))) Gates gate[4];                   // by the chunk's number modulo 4

  int64_t unit;
  int part;
  if (!gdr_block(blockIdx.x, p.n_seq * p.Hv, p.dv / 16, &unit, &part)) return;
  const int h = (int)(unit % p.Hv), kh = h / (p.Hv / p.Hk);
  const int64_t s = by_length(p, unit / p.Hv);
  unit = s * p.Hv + h;
  const GdrSeq seq = gdr_seq(p, s);
  const int64_t nc = seq.n_chunks;
  const int lane = threadIdx.x & 63, li = lane & 15, g = lane >> 4;
  const int wave = wave_id() & 3;
  const int col = 16 * part + li;
  const int r0 = 16 * wave + 4 * g;
  const int last_rows = (int)(seq.len - (nc - 1) * kGdrChunk);
  const bool owner = wave * RT < DK / 16;
  const int first_tile = owner ? wave * RT : 0;
  const int64_t blk0 = seq.slot0 * p.Hv + h;

  if (wave_id() < 4) {
    floatx4 S[RT];
#pragma unroll
    for (int m = 0; m < RT; ++m) {
      S[m] = floatx4{};
      if (owner && p.dSf) {
        const auto at = global_in<float>(p.dSf) + unit * p.dk * p.dv + (16 * (wave * RT + m) + 4 * g) * p.dv + col;
#pragma unroll
        for (int r = 0; r < 4; ++r) S[m][r] = at[r * p.dv];
      }
    }
    auto put_state = [&]() {
#pragma unroll
      for (int m = 0; m < RT; ++m) {
        const int t = wave * RT + m;
        if (owner) put_op<3>(sf + (t >> 1) * kOp3, t & 1, li, g, S[m], T{});
      }
    };
    put_state();
    auto walk = [&](auto both) {
      constexpr int TS = decltype(both)::value ? 2 : 1;   // T^T of wavefronts 0 and 1 reaches into both steps
      // the last chunk first, then downwards
      RowLoads<T, DK> kr(global_in<T>(p.k) + seq.row * p.sk.b + kh * p.sk.h + (seq.t0 + (nc - 1) * kGdrChunk) * p.sk.t, wave, lane, last_rows, p.sk.t);
      auto tp = as_global((const char*)p.ws_tt) + (blk0 + (nc - 1) * p.Hv) * kTriFrags * kOp3 + upper_frag(wave, wave < 2 ? 0 : 1) * kOp3;
      int64_t k_at = nc - 1, t_at = nc - 1;
      In kf[KS];
      Op3 tt[TS];
      auto load_k = [&]() {
        kr.load(k_at == nc - 1);
        const int64_t more = mask_of(k_at > 0);
        k_at -= more & 1;
        kr.from -= more & (int64_t)(kGdrChunk * p.sk.t);
      };
      auto turn_k = [&]() {
        kl.leave(kr.v, 16 * wave, lane);
        compiler_fence();
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) kf[ks] = kl.row_frag(wave, ks, lane);
      };
      auto load_tt = [&]() {
#pragma unroll
        for (int ks = 0; ks < TS; ++ks) tt[ks] = load_frag<Op3>(tp + ks * kOp3, lane);
        const int64_t more = mask_of(t_at > 0);
        t_at -= more & 1;
        tp -= more & (int64_t)(p.Hv * (kTriFrags * kOp3));
      };
      auto step = [&](int64_t c, int n) {
        const Gates& gt = gate[c & 3];
        load_k();
        Op3 sb[KS];
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) sb[ks] = load_frag<Op3>((const char*)sf + ks * kOp3, lane);
        const floatx4 first = ld4f((const float*)&x0[(wave * 64 + lane) * 4]), eta = ld4f((const float*)gt.eta + r0);
        floatx4 X = mma_steps(kf, sb, floatx4{});
#pragma unroll
        for (int r = 0; r < 4; ++r) X[r] = r0 + r < n ? eta[r] * X[r] + first[r] : 0.f;
        put_op<3>(xf + (wave >> 1) * kOp3, wave & 1, li, g, X, T{});
        block_barrier();

        Op3 xb[TS];
#pragma unroll
        for (int ks = 0; ks < TS; ++ks) xb[ks] = load_frag<Op3>((const char*)xf + (ks + 2 - TS) * kOp3, lane);
        const floatx4 gam = ld4f((const float*)gt.gam + r0), beta = ld4f((const float*)gt.beta + r0);
        const float last = gt.gam[63];
        In kt[RT][2];
#pragma unroll
        for (int m = 0; m < RT; ++m) {
          const floatx4 add = ld4f((const float*)&d0[((first_tile + m) * 64 + lane) * 4]);
          S[m] = S[m] * last + add;
#pragma unroll
          for (int ks = 0; ks < 2; ++ks) kt[m][ks] = kl.transposed(first_tile + m, ks, lane);
        }
        const floatx4 dU = mma_steps(tt, xb, floatx4{});
        load_tt();
        put_op<3>(ef + (wave >> 1) * kOp3, wave & 1, li, g, -(gam * beta) * dU, T{});
        ut.put_tile(li, r0, dU);
        block_barrier();

        const Op3 eb[2] = {load_frag<Op3>((const char*)ef, lane), load_frag<Op3>((const char*)ef + kOp3, lane)};
#pragma unroll
        for (int m = 0; m < RT; ++m) S[m] = mma_steps(kt[m], eb, S[m]);
        turn_k();
        put_state();
        block_barrier();
      };
      if (nc > 0) {
        load_k();
        load_tt();
        turn_k();
      }
      block_barrier();
      block_barrier();
      block_barrier();
      for (int64_t c = nc - 1; c >= 0; --c) step(c, c == nc - 1 ? last_rows : kGdrChunk);
    };
    if (wave < 2) walk(std::true_type{});
    else walk(std::false_type{});
    if (p.dS0 && owner) {
#pragma unroll
      for (int m = 0; m < RT; ++m) {
        const auto at = global_out<float>(p.dS0) + unit * p.dk * p.dv + (16 * (wave * RT + m) + 4 * g) * p.dv + col;
#pragma unroll
        for (int r = 0; r < 4; ++r) at[r * p.dv] = S[m][r];
      }
    }
    return;
  }

  // wavefronts 4-7: dO and the gates are fetched two chunks ahead of the chain and turned in LDS, what they make
  // is ready one chunk ahead
  auto serve = [&](auto both) {
    constexpr int TS = decltype(both)::value ? 2 : 1;
    const int tid = threadIdx.x & 255;
    In ox, fx, f2;
    float gx = 0.f;
    Op3 pm[TS];
    RowLoads<T, DK> qr(global_in<T>(p.q) + seq.row * p.sq.b + kh * p.sq.h + (seq.t0 + (nc - 1) * kGdrChunk) * p.sq.t, wave, lane, last_rows, p.sq.t);
    int64_t at = nc - 1, pat = nc - 1, qat = nc - 1;   // the chunk that is fetched next, and whose P and Q are loaded next
    auto dop = global_in<T>(p.dO) + seq.row * p.sdo.b + h * p.sdo.h + (seq.t0 + at * kGdrChunk) * p.sdo.t + 16 * part;
    auto gp = global_in<float>(p.ws_gate) + (blk0 + at * p.Hv) * kGateFloats + (wave < 3 ? wave : 0) * 64;
    auto pp = as_global((const char*)p.ws_p) + ((blk0 + at * p.Hv) * kTriFrags + upper_frag(wave, TS == 2 ? 0 : 1)) * kOp3;
    // of the chunk the chain is at
    const int64_t s_plane = p.dk * p.dv, f_plane = kGdrChunk * p.dv;
    auto fp = global_in<T>(p.ws_f) + (blk0 + at * p.Hv) * kKept<T> * f_plane + part * (kGdrChunk * 16);
    auto sp = global_out<T>(p.ws_ds) + (blk0 + at * p.Hv) * kKept<T> * s_plane + part * (DK * 16);
    auto ep = global_out<T>(p.ws_e) + (blk0 + at * p.Hv) * f_plane + part * (kGdrChunk * 16);
    auto dvp = global_out<T>(p.dv_) + seq.row * p.sdv.b + h * p.sdv.h + (seq.t0 + at * kGdrChunk) * p.sdv.t + 16 * part;
    auto dbp = global_out<float>(p.ws_db) + ((blk0 + at * p.Hv) * (p.dv / 16) + part) * kGdrChunk;
    // wavefronts 4 and 5 move dO, wavefronts 6 and 7 F, dU and the gradients that are made of them: a lane has
    // half a token's columns
    const int tid2 = tid & 127, row = tid2 >> 1;
    const LaneRow orow(row, last_rows, p.sdo.t, 8 * (tid & 1), sizeof(T));
    const uint32_t frow = (uint32_t)(tid2 * 8 * sizeof(T));
    const uint32_t vrow = (uint32_t)((row * p.sdv.t + 8 * (tid2 & 1)) * sizeof(T));
    auto fetch = [&]() {
      if (wave < 2) ox = load_row8(lane_at(dop, orow.of(at == nc - 1)));
      if (wave < 3) gx = *lane_at(gp, lane * 4);
      const int64_t more = mask_of(at > 0);
      at -= more & 1;
      dop -= more & (int64_t)(kGdrChunk * p.sdo.t);
      gp -= more & (int64_t)(p.Hv * kGateFloats);
    };
    auto leave = [&](int64_t c) {
      if (wave < 2) ot.put_row(tid, ox);
      if (wave < 3) (wave == 0 ? gate[c & 3].gam : wave == 1 ? gate[c & 3].eta : gate[c & 3].beta)[lane] = gx;
    };
    auto load_p = [&]() {
#pragma unroll
      for (int ks = 0; ks < TS; ++ks) pm[ks] = load_frag<Op3>(pp + ks * kOp3, lane);
      const int64_t more = mask_of(pat > 0);
      pat -= more & 1;
      pp -= more & (int64_t)(p.Hv * (kTriFrags * kOp3));
    };
    auto load_q = [&]() {
      qr.load(qat == nc - 1);
      const int64_t more = mask_of(qat > 0);
      qat -= more & 1;
      qr.from -= more & (int64_t)(kGdrChunk * p.sq.t);
    };
    auto load_f = [&](int64_t c) {
      if (wave >= 2) {
        fx = load_row8(lane_at(fp, frow));
        if constexpr (kKept<T> == 2) f2 = load_row8(lane_at(fp + f_plane, frow));
      }
      fp -= mask_of(c > 0) & (int64_t)(p.Hv * kKept<T> * f_plane);
    };
    auto spread = [&](int64_t c) {       // dO of chunk c as operands, and its Q
      const int n = c == nc - 1 ? last_rows : kGdrChunk;
      const floatx4 gam = p.scale * ld4f((const float*)gate[c & 3].gam + r0);
      ql.leave(qr.v, 16 * wave, lane);
      load_q();
      floatx4 x = ot.tile(li, r0);
#pragma unroll
      for (int r = 0; r < 4; ++r) x[r] = r0 + r < n ? x[r] : 0.f;
      put_op<1>(of + (wave >> 1) * kIn, wave & 1, li, g, x, T{});
      put_op<3>(gf + (wave >> 1) * kOp3, wave & 1, li, g, gam * x, T{});
    };
    // x0 and d0 are read by the chain before this chunk's second barrier and written after it
    floatx4 X, D[RT];
    auto products = [&]() {
      In qt[RT][2];
#pragma unroll
      for (int m = 0; m < RT; ++m)
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) qt[m][ks] = ql.transposed(first_tile + m, ks, lane);
      X = mma(pm[TS - 1], load_frag<In>((const char*)of + kIn, lane), floatx4{});
      if constexpr (TS == 2) X = mma(pm[0], load_frag<In>((const char*)of, lane), X);
      const Op3 gb[2] = {load_frag<Op3>((const char*)gf, lane), load_frag<Op3>((const char*)gf + kOp3, lane)};
#pragma unroll
      for (int m = 0; m < RT; ++m) {
        D[m] = mma_steps(qt[m], gb, floatx4{});
        settle(D[m]);
      }
      settle(X);
    };
    auto leave_products = [&]() {
      *reinterpret_cast<floatx4*>(&x0[(wave * 64 + lane) * 4]) = X;
#pragma unroll
      for (int m = 0; m < RT; ++m)
        if (owner) *reinterpret_cast<floatx4*>(&d0[((wave * RT + m) * 64 + lane) * 4]) = D[m];
    };
    // dU as the chain has left it: the gradient of v, and beta's over these columns
    auto finish = [&](int64_t c) {
      const int n = c == nc - 1 ? last_rows : kGdrChunk;
      if (wave >= 2) {
        const float b = gate[c & 3].beta[row];
        const float8v dU = ut.row(tid2);
        T f8[8];
        __builtin_memcpy(f8, &fx, sizeof(fx));
        float x = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) x += dU[e] * value(f8[e]);
        if constexpr (kKept<T> == 2) {
          T g8[8];
          __builtin_memcpy(g8, &f2, sizeof(f2));
#pragma unroll
          for (int e = 0; e < 8; ++e) x += dU[e] * value(g8[e]);
        }
        x += __shfl_xor(x, 1);
        if ((tid & 1) == 0) *lane_at(dbp, row * 4) = x;
        if constexpr (sizeof(T) == 2) {   // dE in two planes, the first of which is the gradient itself
          const Planes<2> dE = make_op<2>(b * dU, T{});
          if (row < n) *repoint<bf16x8>(lane_at(dvp, vrow)) = dE.p[0];
          *repoint<bf16x8>(lane_at(ep, frow)) = dE.p[1];
        } else if (row < n) {
          store_row4(lane_at(dvp, vrow), b * floatx4{dU[0], dU[1], dU[2], dU[3]});
          store_row4(lane_at(dvp, vrow + 4 * sizeof(T)), b * floatx4{dU[4], dU[5], dU[6], dU[7]});
        }
      }
      ep -= p.Hv * f_plane;
      dvp -= kGdrChunk * p.sdv.t;
      dbp -= p.Hv * (p.dv / 16 * kGdrChunk);
    };
    if (nc > 0) {
      fetch();
      load_p();
      load_q();
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
      load_p();
      leave(nc - 2);
      fetch();
    }
    block_barrier();
    for (int64_t c = nc - 1; c >= 0; --c) {
      // dS at this chunk's end; what the chain needs of the next one
      write_rows<T>(sf, kOp3, DK, sp, s_plane, tid);
      sp -= p.Hv * kKept<T> * s_plane;
      if (c > 0) spread(c - 1);
      block_barrier();
      if (c > 0) products();
      block_barrier();
      if (c > 0) {
        leave_products();
        load_p();
      }
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

template <typename T, int DK>
hipError_t launch_scan(const GdrParams& p, hipStream_t s, int kind) {
  const dim3 grid((unsigned)gdr_blocks(p.n_seq * p.Hv, p.dv / 16));
  if (kind == 0) hipLaunchKernelGGL((gdr_scan_kernel<T, DK, false>), grid, dim3(512), 0, s, p);
  else if (kind == 1) hipLaunchKernelGGL((gdr_scan_kernel<T, DK, true>), grid, dim3(512), 0, s, p);
  else hipLaunchKernelGGL((gdr_rscan_kernel<T, DK>), grid, dim3(512), 0, s, p);
  return hipGetLastError();
}

template <typename T>
hipError_t launch_t(const GdrParams& p, hipStream_t s, int kind) {
  switch (p.dk) {
    case 32: return launch_scan<T, 32>(p, s, kind);
    case 64: return launch_scan<T, 64>(p, s, kind);
    default: return launch_scan<T, 128>(p, s, kind);
  }
}

hipError_t launch_kind(const GdrParams& p, hipStream_t s, int kind) {
  return p.dtype == KDA_DTYPE_BF16 ? launch_t<uint16_t>(p, s, kind) : launch_t<float>(p, s, kind);
}

}  // namespace

hipError_t launch_gdr_scan(const GdrParams& p, hipStream_t s, bool states) { return launch_kind(p, s, states ? 1 : 0); }
hipError_t launch_gdr_rscan(const GdrParams& p, hipStream_t s) { return launch_kind(p, s, 2); }

}  // namespace kda
