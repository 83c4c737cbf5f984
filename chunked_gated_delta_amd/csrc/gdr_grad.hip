// Gradients of the head-gated delta rule from each chunk's entering state S, F = U / beta, the state's
// adjoint dS at the chunk's end and dE (the gradient of v): one workgroup per (chunk, key head), the
// value heads that share the key head one after another.
//
// A wavefront owns 16 tokens and half of the channels and forms the transposed gradients (channels x
// tokens), so a lane holds one token and 4 consecutive channels.  bf16: the workgroup asks for all its operands
// at once (240 KiB at dk = dv = 128: one workgroup's whole traffic in flight), in the order it uses them, and
// shares them in LDS, the states a plane at a time; K^T and Q^T are transposing LDS reads.  With dO' = scale dO and
// D_rj = e^{G_r - G_j}:
//   dP = lower(dO' U^T . D)   dA = -strict_lower(dE U^T . D)
//   dq_r  =  gam_r S dO'_r + sum_j dP_rj k_j
//   dk_r  = -gam_r S dE_r  + sum_j dA_rj k_j                                    (as a row: reads)
//         +  eta_r dS U_r  + sum_r' dA_r'r k_r' + sum_r' dP_r'r q_r'            (as a column: writes)
//   dG_r  = q_r . dq_r + k_r . dk_r(row) - k_r . dk_r(column),   dG_last += sum_r k_r . eta_r dS U_r + e^{G_last} <S, dS>
//   dg_t  = sum_{r >= t} dG_r
// The second identity gives the log-decay's gradient from the accumulators that are there anyway.  S, dS, F and
// dE come in two bf16 planes, dP and dA are made of two (off by 2^-17): with one plane of each, 2x4096 tokens' kernel
// took 164 us, but dk and dw were off by up to 3.6e-3 where the rounding of the results is 1.7e-3.
//
// 2 x 4096 tokens, 16 heads of 128 x 128 in bf16: 211 to 227 us for 0.6 GB.  At 128 x 128 all 256 registers are used and 25
// more spilled (22 in fp32); no smaller size spills.  One workgroup fills a compute unit's LDS, so half
// of its cycles wait for the loads (all compute units ask at once) and the other half use none of the bandwidth; where
// value heads share a key head, the next one's operands are asked for before the last sums of the one before.
#include <type_traits>

#include "gdr_internal.h"

namespace kda {

namespace {

template <int DK, int DV>
__global__ __launch_bounds__(512) void gdr_grad_kernel(GdrParams p) {
  using T = uint16_t;
  constexpr int KV = DV / 32, MT = DK / 16, MH = MT / 2;   // MH: channel tiles of a wavefront
  constexpr int kOp = op_frag<T, 2>(), kLd = DV + 8;
  constexpr int kRow8 = DV / 8;                            // 16-byte pieces of a row
  constexpr int kTok = 64 * kRow8 / 512 ? 64 * kRow8 / 512 : 1;   // pieces a thread moves of 64 rows,
  constexpr int kSt = DK * kRow8 / 512 ? DK * kRow8 / 512 : 1;    // of DK rows,
  constexpr int kCh = 64 * (DK / 8) / 512 ? 64 * (DK / 8) / 512 : 1;   // and of K or Q,
  constexpr bool kAllTok = 64 * kRow8 % 512 == 0, kAllSt = DK * kRow8 % 512 == 0, kAllCh = 64 * (DK / 8) % 512 == 0;   // all of them
  constexpr int kTri = 4 * 8 * kOp, kXBytes = 5 * 64 * kLd * 2 > kTri ? 5 * 64 * kLd * 2 : kTri;
  // F, dO and dE (F and dE in two planes); then the triangular factors: per token tile 2 steps of dP and dA over j,
  // 2 of each over r
  __shared__ __attribute__((aligned(16))) char xs[kXBytes];
  __shared__ __attribute__((aligned(16))) T sl[DK * kLd];  // a plane of S, then of dS
  __shared__ __attribute__((aligned(16))) Rows<T, DK> kl, ql;
  __shared__ __attribute__((aligned(16))) float ghi[64], glo[64], bet[64];
  __shared__ double dG[2][64], extra[8];
  T* fl = reinterpret_cast<T*>(xs);
  T* f2l = fl + 64 * kLd;
  T* ol = f2l + 64 * kLd;
  T* el = ol + 64 * kLd;
  T* e2l = el + 64 * kLd;

  GdrSeq seq;
  int64_t chunk;
  const int64_t slot = blockIdx.x;
  if (!gdr_find(p, slot, &seq, &chunk)) return;
  const int kh = blockIdx.y, grp = p.Hv / p.Hk;
  int tid = threadIdx.x;
  const int tile = wave_id() & 3, half = wave_id() >> 2;   // token tile; half of the channels
  const int64_t t0 = seq.t0 + chunk * kGdrChunk, left = seq.len - chunk * kGdrChunk;
  const int n = left < kGdrChunk ? (int)left : kGdrChunk;
  char* mine = xs + tile * 8 * kOp;

  floatx4 dq[MH], dk[MH];
#pragma unroll
  for (int m = 0; m < MH; ++m) dq[m] = dk[m] = floatx4{};

  for (int hg = 0; hg < grp; ++hg) {
    // said anew for every head: addresses that the loop does not change would otherwise be kept in registers
    // by the dozen
    asm volatile("" : "+v"(tid));
    const int lane = tid & 63, li = lane & 15, g = lane >> 4;
    const int tok = 16 * tile + li;                        // this lane's token
    const int h = kh * grp + hg;
    const int64_t blk = slot * p.Hv + h;
    const auto gate = global_in<float>(p.ws_gate) + blk * kGateFloats;
    const auto F = global_in<T>(p.ws_f) + blk * 2 * kGdrChunk * DV;
    const auto E2 = global_in<T>(p.ws_e) + blk * kGdrChunk * DV;
    const auto St = global_in<T>(p.ws_s) + blk * 2 * DK * DV;
    const auto dSt = global_in<T>(p.ws_ds) + blk * 2 * DK * DV;
    const auto dO = global_in<T>(p.dO) + seq.row * p.sdo.b + h * p.sdo.h + t0 * p.sdo.t;
    const auto dE = global_in<T>(p.dv_) + seq.row * p.sdv.b + h * p.sdv.h + t0 * p.sdv.t;
    // everything is asked for at once, in the order of its use: loads are waited for in the order they were asked
    const float gates[3] = {gate[kGateHi + lane], gate[kGateLo + lane], gate[kGateBeta + lane]};
    const float gam = gate[kGateGam + tok], eta = gate[kGateEta + tok], last = gate[kGateLast];
    bf16x8 fx[kTok], f2[kTok], ox[kTok], ex[kTok], e2[kTok], sx[kSt], s2[kSt], dx[kSt], d2[kSt], kx[kCh], qx[kCh];
#pragma unroll
    for (int i = 0; i < kTok; ++i) {
      const int at = tid + 512 * i, r = at / kRow8, c0 = at % kRow8 * 8;
      fx[i] = f2[i] = ox[i] = ex[i] = e2[i] = bf16x8{};
      if (kAllTok || at < 64 * kRow8) {
        fx[i] = load_row8(F + at * 8);
        f2[i] = load_row8(F + kGdrChunk * DV + at * 8);
      }
      if (r < n && (kAllTok || at < 64 * kRow8)) {
        ox[i] = load_row8(dO + r * p.sdo.t + c0);
        ex[i] = load_row8(dE + r * p.sdv.t + c0);
      }
      if (at % 128 / 2 < n && (kAllTok || at < 64 * kRow8)) e2[i] = load_row8(E2 + at * 8);
    }
    if (hg == 0) {   // K and Q, zeros behind the sequence's end
#pragma unroll
      for (int i = 0; i < kCh; ++i) {
        const int at = tid + 512 * i, r = at / (DK / 8), c0 = at % (DK / 8) * 8;
        kx[i] = qx[i] = bf16x8{};
        if (r < n) {
          kx[i] = load_row8(global_in<T>(p.k) + seq.row * p.sk.b + kh * p.sk.h + (t0 + r) * p.sk.t + c0);
          qx[i] = load_row8(global_in<T>(p.q) + seq.row * p.sq.b + kh * p.sq.h + (t0 + r) * p.sq.t + c0);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kSt; ++i) {
      const int at = tid + 512 * i;
      sx[i] = bf16x8{};
      if (kAllSt || at < DK * kRow8) sx[i] = load_row8(St + at * 8);
    }
#pragma unroll
    for (int i = 0; i < kSt; ++i) {
      const int at = tid + 512 * i;
      s2[i] = dx[i] = d2[i] = bf16x8{};
      if (kAllSt || at < DK * kRow8) {
        s2[i] = load_row8(St + DK * DV + at * 8);
        dx[i] = load_row8(dSt + at * 8);
        d2[i] = load_row8(dSt + DK * DV + at * 8);
      }
    }
    if (hg > 0) block_barrier();   // the head before has used what lies in LDS
    if (tid < 64) {
      ghi[tid] = gates[0];
      glo[tid] = gates[1];
      bet[tid] = gates[2];
    }
    // piece `at` of a matrix kept as 16 columns after the other, `rows` of 16 values each
    auto at_part = [&](T* base, int at, int rows) {
      return reinterpret_cast<bf16x8*>(base + at % (2 * rows) / 2 * kLd + at / (2 * rows) * 16 + (at & 1) * 8);
    };
    auto at_row = [&](T* base, int at) { return reinterpret_cast<bf16x8*>(base + at / kRow8 * kLd + at % kRow8 * 8); };
#pragma unroll
    for (int i = 0; i < kTok; ++i) {
      const int at = tid + 512 * i;
      if (kAllTok || at < 64 * kRow8) {
        *at_part(fl, at, 64) = fx[i];
        *at_part(f2l, at, 64) = f2[i];
        *at_row(ol, at) = ox[i];
        *at_row(el, at) = ex[i];
        *at_part(e2l, at, 64) = e2[i];
      }
    }
    auto put_plane = [&](const bf16x8 (&x)[kSt]) {
#pragma unroll
      for (int i = 0; i < kSt; ++i)
        if (kAllSt || tid + 512 * i < DK * kRow8) *at_part(sl, tid + 512 * i, DK) = x[i];
    };
    put_plane(sx);
    if (hg == 0) {
#pragma unroll
      for (int i = 0; i < kCh; ++i) {
        const int at = tid + 512 * i, row = at / (DK / 8), c0 = at % (DK / 8) * 8;
        if (kAllCh || row < 64) {
          kl.put8(row, c0, kx[i]);
          ql.put8(row, c0, qx[i]);
        }
      }
    }
    block_barrier();

    auto rows = [&](const T* base, int t, int kv) { return load_row8(base + (16 * t + li) * kLd + 32 * kv + 8 * g); };
    // this wavefront's own tokens
    auto own = [&](const T* base, bf16x8 (&x)[KV]) {
#pragma unroll
      for (int kv = 0; kv < KV; ++kv) x[kv] = rows(base, tile, kv);
    };
    bf16x8 fo[KV], fo2[KV], oo[KV], eo[KV], eo2[KV];
    own(ol, oo);
    own(el, eo);
    own(e2l, eo2);
    double dg = 0.0, write = 0.0, hold = 0.0;
    // S dO, S dE and dS U of this wavefront's channels, a plane of the states at a time
    floatx4 a[MH], b[MH], c[MH];
#pragma unroll
    for (int mm = 0; mm < MH; ++mm) {
      a[mm] = b[mm] = c[mm] = floatx4{};
#pragma unroll
      for (int kv = 0; kv < KV; ++kv) {
        const bf16x8 st = rows(sl, half * MH + mm, kv);
        a[mm] = mma(st, oo[kv], a[mm]);
        b[mm] = mma(st, eo2[kv], b[mm]);
        b[mm] = mma(st, eo[kv], b[mm]);
      }
    }
    block_barrier();
    put_plane(s2);
    block_barrier();
#pragma unroll
    for (int mm = 0; mm < MH; ++mm)
#pragma unroll
      for (int kv = 0; kv < KV; ++kv) {
        const bf16x8 st = rows(sl, half * MH + mm, kv);
        a[mm] = mma(st, oo[kv], a[mm]);
        b[mm] = mma(st, eo[kv], b[mm]);
      }
    block_barrier();
    own(fl, fo);
    own(f2l, fo2);
    // <S, dS>: this thread's pieces of both, only now, so that dS may still be on its way
#pragma unroll
    for (int i = 0; i < kSt; ++i) {
      float x = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) x += ((float)sx[i][e] + (float)s2[i][e]) * ((float)dx[i][e] + (float)d2[i][e]);
      hold += x;
    }
    put_plane(dx);
    block_barrier();
#pragma unroll
    for (int mm = 0; mm < MH; ++mm)
#pragma unroll
      for (int kv = 0; kv < KV; ++kv) {
        const bf16x8 st = rows(sl, half * MH + mm, kv);
        c[mm] = mma(st, fo2[kv], c[mm]);
        c[mm] = mma(st, fo[kv], c[mm]);
      }
    block_barrier();
    put_plane(d2);
    block_barrier();
#pragma unroll
    for (int mm = 0; mm < MH; ++mm)
#pragma unroll
      for (int kv = 0; kv < KV; ++kv) c[mm] = mma(rows(sl, half * MH + mm, kv), fo[kv], c[mm]);
    // dP and dA: half 0 over all j <= its tokens r (transposed), half 1 over all r >= its tokens j; tiles that
    // hold none of it stay zeros
    own(ol, oo);   // read again: kept, they would not leave dS's pieces room
    own(el, eo);
    own(e2l, eo2);
    const float ghr = ghi[tok], glr = glo[tok], own_beta = bet[tok];
    floatx4 a4[4], b4[4];
#pragma unroll
    for (int m = 0; m < 4; ++m) a4[m] = b4[m] = floatx4{};
    if (half == 0) {
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        if (m > tile) break;
#pragma unroll
        for (int kv = 0; kv < KV; ++kv) {
          const bf16x8 x = rows(fl, m, kv), x2 = rows(f2l, m, kv);
          a4[m] = mma(x2, oo[kv], a4[m]);
          b4[m] = mma(x2, eo[kv], b4[m]);
          a4[m] = mma(x, oo[kv], a4[m]);
          b4[m] = mma(x, eo2[kv], b4[m]);
          b4[m] = mma(x, eo[kv], b4[m]);
        }
      }
    } else {
#pragma unroll
      for (int m = 3; m >= 0; --m) {
        if (m < tile) break;
#pragma unroll
        for (int kv = 0; kv < KV; ++kv) {
          const bf16x8 x = rows(ol, m, kv), y = rows(el, m, kv), y2 = rows(e2l, m, kv);
          a4[m] = mma(x, fo2[kv], a4[m]);
          b4[m] = mma(y, fo2[kv], b4[m]);
          a4[m] = mma(x, fo[kv], a4[m]);
          b4[m] = mma(y2, fo[kv], b4[m]);
          b4[m] = mma(y, fo[kv], b4[m]);
        }
      }
    }
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      settle(a4[m]);
      settle(b4[m]);
    }
    block_barrier();   // everyone has read F, dO and dE
    auto factors = [&](auto rows_of_tok) {
      constexpr bool kRows = decltype(rows_of_tok)::value;   // o is j of the row tok, or r of the column tok
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        if (kRows ? m <= tile : m >= tile) {
          const floatx4 oh = ld4f((const float*)ghi + 16 * m + 4 * g), ol4 = ld4f((const float*)glo + 16 * m + 4 * g);
          const floatx4 ob = ld4f((const float*)bet + 16 * m + 4 * g);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int o = 16 * m + 4 * g + r;
            const float d = kRows ? (ghr - oh[r]) + (glr - ol4[r]) : (oh[r] - ghr) + (ol4[r] - glr);
            const bool in = kRows ? tok >= o : o >= tok;
            // the fast exponential is off by 2^-23 (1 + |d|): beside two planes' 2^-17 nothing where e^d still counts
            const float w = (kRows ? ob[r] : own_beta) * __expf(in ? d : 0.f);
            a4[m][r] = in ? p.scale * w * a4[m][r] : 0.f;
            b4[m][r] = in && tok != o ? -w * b4[m][r] : 0.f;
          }
        }
        put_op<2>(mine + ((kRows ? 0 : 4) + (m >> 1)) * kOp, m & 1, li, g, a4[m], T{});
        put_op<2>(mine + ((kRows ? 2 : 6) + (m >> 1)) * kOp, m & 1, li, g, b4[m], T{});
      }
    };
    if (half == 0) factors(std::true_type{});
    else factors(std::false_type{});
    block_barrier();

    const float br = bet[tok];
    {   // over j <= r
      Planes<2> pr[2], ar[2];
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        pr[ks] = load_frag<Planes<2>>((const char*)mine + ks * kOp, lane);
        ar[ks] = load_frag<Planes<2>>((const char*)mine + (2 + ks) * kOp, lane);
      }
#pragma unroll
      for (int mm = 0; mm < MH; ++mm) {
        const int m = half * MH + mm;
        const bf16x8 kt[2] = {kl.transposed(m, 0, lane), kl.transposed(m, 1, lane)};
        const floatx4 x = mma_steps(kt, pr, a[mm] * (gam * p.scale)), y = mma_steps(kt, ar, b[mm] * -gam);
        dq[mm] += x;
        dk[mm] += y;
        const u32x2v q2 = *reinterpret_cast<const u32x2v*>(ql.x + tok * ql.kLd + 16 * m + 4 * g);
        const u32x2v k2 = *reinterpret_cast<const u32x2v*>(kl.x + tok * kl.kLd + 16 * m + 4 * g);
        dg += (lo_bf16(q2[0]) * x[0] + hi_bf16(q2[0]) * x[1]) + (lo_bf16(q2[1]) * x[2] + hi_bf16(q2[1]) * x[3]);
        dg += (lo_bf16(k2[0]) * y[0] + hi_bf16(k2[0]) * y[1]) + (lo_bf16(k2[1]) * y[2] + hi_bf16(k2[1]) * y[3]);
      }
    }
    {   // over r >= j
      Planes<2> pc[2], ac[2];
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        pc[ks] = load_frag<Planes<2>>((const char*)mine + (4 + ks) * kOp, lane);
        ac[ks] = load_frag<Planes<2>>((const char*)mine + (6 + ks) * kOp, lane);
      }
#pragma unroll
      for (int mm = 0; mm < MH; ++mm) {
        const int m = half * MH + mm;
        floatx4 x = c[mm] * (eta * br);
        const u32x2v k2 = *reinterpret_cast<const u32x2v*>(kl.x + tok * kl.kLd + 16 * m + 4 * g);
        const floatx4 k4 = {lo_bf16(k2[0]), hi_bf16(k2[0]), lo_bf16(k2[1]), hi_bf16(k2[1])};
        write += (k4[0] * x[0] + k4[1] * x[1]) + (k4[2] * x[2] + k4[3] * x[3]);
        const bf16x8 kt[2] = {kl.transposed(m, 0, lane), kl.transposed(m, 1, lane)};
        const bf16x8 qt[2] = {ql.transposed(m, 0, lane), ql.transposed(m, 1, lane)};
        x = mma_steps(kt, ac, x);
        x = mma_steps(qt, pc, x);
        dk[mm] += x;
        dg -= (k4[0] * x[0] + k4[1] * x[1]) + (k4[2] * x[2] + k4[3] * x[3]);
      }
    }
    // the log-decay's gradient
    dg += __shfl_xor(dg, 16);
    dg += __shfl_xor(dg, 32);
    double sum = write + (double)last * hold;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) sum += __shfl_xor(sum, d);
    if (g == 0) dG[half][tok] = dg;
    if (lane == 0) extra[wave_id()] = sum;
    block_barrier();
    if (wave_id() == 7) {   // while the others ask for the next head's operands
      constexpr int kParts = DV / 16;
      float w_last = 0.f, db_parts[kParts], db_last = 0.f;
      if (lane < n) w_last = get(global_in<T>(p.w) + seq.row * p.sw.b + h * p.sw.h + (t0 + lane) * p.sw.t);
#pragma unroll
      for (int c = 0; c < kParts; ++c) db_parts[c] = global_in<float>(p.ws_db)[(blk * kParts + c) * kGdrChunk + lane];
      double x = dG[0][lane] + dG[1][lane];
      if (lane == 63) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x += extra[i];
      }
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const double dn = __shfl_down(x, d);
        if (lane + d < 64) x += dn;
      }
#pragma unroll
      for (int c = 0; c < kParts; ++c) db_last += db_parts[c];
      if (lane < n) {
        put(global_out<T>(p.dw) + seq.row * p.sdw.b + h * p.sdw.h + (t0 + lane) * p.sdw.t,
            (float)(x * (double)gdr_gate_grad(w_last, p.gate, p.g_min)));
        put(global_out<T>(p.dbeta) + seq.row * p.sdb.b + h * p.sdb.h + (t0 + lane) * p.sdb.t, db_last);
      }
    }
  }

  // whole rows: 8 bytes a lane as they lie here would be written to memory twice over
  block_barrier();   // K and Q are used
  const int lane = tid & 63, g = lane >> 4, tok = 16 * tile + (lane & 15);
#pragma unroll
  for (int mm = 0; mm < MH; ++mm) {
    const int c = 16 * (half * MH + mm) + 4 * g;
    *reinterpret_cast<u32x2v*>(ql.x + tok * ql.kLd + c) = u32x2v{pk_bf16(dq[mm][0], dq[mm][1]), pk_bf16(dq[mm][2], dq[mm][3])};
    *reinterpret_cast<u32x2v*>(kl.x + tok * kl.kLd + c) = u32x2v{pk_bf16(dk[mm][0], dk[mm][1]), pk_bf16(dk[mm][2], dk[mm][3])};
  }
  block_barrier();
#pragma unroll
  for (int i = 0; i < kCh; ++i) {
    const int at = tid + 512 * i, row = at / (DK / 8), c0 = at % (DK / 8) * 8;
    if (row < n) {
      *repoint<bf16x8>(global_out<T>(p.dq) + seq.row * p.sdq.b + kh * p.sdq.h + (t0 + row) * p.sdq.t + c0) = load_row8(ql.x + row * ql.kLd + c0);
      *repoint<bf16x8>(global_out<T>(p.dk_) + seq.row * p.sdk.b + kh * p.sdk.h + (t0 + row) * p.sdk.t + c0) = load_row8(kl.x + row * kl.kLd + c0);
    }
  }
}

// fp32 inputs: the same sums, a lane's operands straight from memory, since three 64-row tiles and a state in fp32
// would not fit LDS beside K and Q.  5 sequences of 0 to 447 tokens, 4 heads of 64 x 128: 69 us, of which most are the
// trips to memory of 30 workgroups.
template <int DK, int DV>
__global__ __launch_bounds__(512) void gdr_grad_f32_kernel(GdrParams p) {
  using T = float;
  using In = Frags<float>::In;
  using Op = float8v;
  constexpr int KV = DV / 32, MH = DK / 32;   // MH: channel tiles of a wavefront
  constexpr int kOpFrag = op_frag<T, 2>();
  __shared__ __attribute__((aligned(16))) char tri[4][4 * kOpFrag];   // a token tile's dP and dA, two steps each
  __shared__ __attribute__((aligned(16))) Rows<T, DK> kl, ql;
  __shared__ float ghi[64], glo[64], bet[64];
  __shared__ double dG[2][64], extra[8];

  GdrSeq seq;
  int64_t chunk;
  const int64_t slot = blockIdx.x;
  if (!gdr_find(p, slot, &seq, &chunk)) return;
  const int kh = blockIdx.y, grp = p.Hv / p.Hk;
  int lane = threadIdx.x & 63;
  const int wave = wave_id() & 3, half = wave_id() >> 2;   // token tile; half of the channels
  const int64_t t0 = seq.t0 + chunk * kGdrChunk, left = seq.len - chunk * kGdrChunk;
  const int n = left < kGdrChunk ? (int)left : kGdrChunk;
  char* dp_f = tri[wave];                         // dP (transposed, then as it is)
  char* da_f = tri[wave] + 2 * kOpFrag;

  for (int i = threadIdx.x; i < 64 * DK / 8; i += 512) {   // K and Q, zeros behind the sequence's end
    const int r = i / (DK / 8), c0 = i % (DK / 8) * 8;
    In a, b;
    zero_frag(a);
    zero_frag(b);
    if (r < n) {
      a = load_row8(global_in<T>(p.k) + seq.row * p.sk.b + kh * p.sk.h + (t0 + r) * p.sk.t + c0);
      b = load_row8(global_in<T>(p.q) + seq.row * p.sq.b + kh * p.sq.h + (t0 + r) * p.sq.t + c0);
    }
    kl.put8(r, c0, a);
    ql.put8(r, c0, b);
  }

  floatx4 dq[MH], dk[MH];
#pragma unroll
  for (int m = 0; m < MH; ++m) dq[m] = dk[m] = floatx4{};

  for (int hg = 0; hg < grp; ++hg) {
    asm volatile("" : "+v"(lane));   // said anew for every head, as above
    const int li = lane & 15, g = lane >> 4, tok = 16 * wave + li;   // tok: this lane's token
    const int h = kh * grp + hg;
    const int64_t blk = slot * p.Hv + h;
    const auto gate = global_in<float>(p.ws_gate) + blk * kGateFloats;
    if (wave_id() == 0) {
      ghi[lane] = gate[kGateHi + lane];
      glo[lane] = gate[kGateLo + lane];
      bet[lane] = gate[kGateBeta + lane];
    }
    const float gam = gate[kGateGam + tok], eta = gate[kGateEta + tok], last = gate[kGateLast];
    const auto F = global_in<T>(p.ws_f) + blk * kGdrChunk * DV + 8 * (g & 1);   // 16 columns after the other
    const auto St = global_in<T>(p.ws_s) + blk * DK * DV + 8 * (g & 1);
    const auto dSt = global_in<T>(p.ws_ds) + blk * DK * DV + 8 * (g & 1);
    const auto dO = global_in<T>(p.dO) + seq.row * p.sdo.b + h * p.sdo.h + t0 * p.sdo.t + 8 * g;
    const auto dE = global_in<T>(p.dv_) + seq.row * p.sdv.b + h * p.sdv.h + t0 * p.sdv.t + 8 * g;
    auto f_frag = [&](int tile, int kv) { return load_row8(F + ((2 * kv + (g >> 1)) * kGdrChunk + 16 * tile + li) * 16); };
    auto rows_of = [&](GlobalPtr<const T> base, int64_t st, int tile, int kv) {
      const int r = 16 * tile + li;   // rows behind the end: the last one's, as zeros
      const In x = load_row8(base + (int64_t)min(r, n - 1) * st + 32 * kv);
      In zero;
      zero_frag(zero);
      return r < n ? x : zero;
    };
    In fo[KV], oo[KV], eo[KV];   // this wavefront's own tokens
#pragma unroll
    for (int kv = 0; kv < KV; ++kv) {
      fo[kv] = f_frag(wave, kv);
      oo[kv] = rows_of(dO, p.sdo.t, wave, kv);
      eo[kv] = rows_of(dE, p.sdv.t, wave, kv);
    }
    __syncthreads();
    const float ghr = ghi[tok], glr = glo[tok], br = bet[tok];

    // rows: dP_rj and dA_rj of this tile's r over all j <= r, as B operands over j; every other tile of j
#pragma unroll
    for (int mm = 0; mm < 2; ++mm) {
      const int m = 2 * mm + half;
      if (m > (wave | 1)) continue;
      floatx4 a = {}, b = {};
      if (m <= wave) {
        In f[KV];
#pragma unroll
        for (int kv = 0; kv < KV; ++kv) f[kv] = f_frag(m, kv);
        __builtin_amdgcn_sched_barrier(0);   // a tile's loads go out together: one by one, each takes a trip to memory
#pragma unroll
        for (int kv = 0; kv < KV; ++kv) {
          a = mma(f[kv], oo[kv], a);
          b = mma(f[kv], eo[kv], b);
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int j = 16 * m + 4 * g + r;
          const float d = tok >= j ? bet[j] * expf((ghr - ghi[j]) + (glr - glo[j])) : 0.f;
          a[r] = tok >= j ? p.scale * d * a[r] : 0.f;
          b[r] = tok > j ? -d * b[r] : 0.f;
        }
      }
      put_op<2>(dp_f + mm * kOpFrag, half, li, g, a, T{});
      put_op<2>(da_f + mm * kOpFrag, half, li, g, b, T{});
    }
    __syncthreads();
    double dg = 0.0, write = 0.0, hold = 0.0;
#pragma unroll
    for (int i = 0; i < MH; ++i) {
      const int m = half * MH + i;
      floatx4 a = {}, b = {};
      float ss = 0.f;
      In st[KV], dst[KV];
#pragma unroll
      for (int kv = 0; kv < KV; ++kv) {
        st[kv] = load_row8(St + ((2 * kv + (g >> 1)) * DK + 16 * m + li) * 16);
        dst[kv] = load_row8(dSt + ((2 * kv + (g >> 1)) * DK + 16 * m + li) * 16);
      }
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int kv = 0; kv < KV; ++kv) {
#pragma unroll
        for (int e = 0; e < 8; ++e) ss += (float)st[kv][e] * (float)dst[kv][e];
        a = mma(st[kv], oo[kv], a);
        b = mma(st[kv], eo[kv], b);
      }
      asm volatile("" : "+v"(ss));   // now: put off to the end, it would keep every row of S and dS till then
      hold += (m & 3) == wave ? ss : 0.f;   // <S, dS>: every row tile once
      a *= gam * p.scale;
      b *= -gam;
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        if (ks > wave / 2) continue;
        const In x = kl.transposed(m, ks, lane);
        a = mma(x, load_frag<Op>(dp_f + ks * kOpFrag, lane), a);
        b = mma(x, load_frag<Op>(da_f + ks * kOpFrag, lane), b);
      }
      settle(a);
      settle(b);
      dq[i] += a;
      dk[i] += b;
      const floatx4 q4 = ld4f(ql.x + tok * ql.kLd + 16 * m + 4 * g), k4 = ld4f(kl.x + tok * kl.kLd + 16 * m + 4 * g);
#pragma unroll
      for (int r = 0; r < 4; ++r) dg += (double)q4[r] * (double)a[r] + (double)k4[r] * (double)b[r];
    }
    __syncthreads();

    // columns: dP_rj and dA_rj of this tile's j over all r >= j, as B operands over r
#pragma unroll
    for (int mm = 0; mm < 2; ++mm) {
      const int m = 2 * mm + half;
      if (m < (wave & 2)) continue;
      floatx4 a = {}, b = {};
      if (m >= wave) {
        In od[KV], ed[KV];
#pragma unroll
        for (int kv = 0; kv < KV; ++kv) {
          od[kv] = rows_of(dO, p.sdo.t, m, kv);
          ed[kv] = rows_of(dE, p.sdv.t, m, kv);
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int kv = 0; kv < KV; ++kv) {
          a = mma(od[kv], fo[kv], a);
          b = mma(ed[kv], fo[kv], b);
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int i = 16 * m + 4 * g + r;
          const float d = i >= tok ? br * expf((ghi[i] - ghr) + (glo[i] - glr)) : 0.f;
          a[r] = i >= tok ? p.scale * d * a[r] : 0.f;
          b[r] = i > tok ? -d * b[r] : 0.f;
        }
      }
      put_op<2>(dp_f + mm * kOpFrag, half, li, g, a, T{});
      put_op<2>(da_f + mm * kOpFrag, half, li, g, b, T{});
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < MH; ++i) {
      const int m = half * MH + i;
      floatx4 a = {};
      In dst[KV];
#pragma unroll
      for (int kv = 0; kv < KV; ++kv) dst[kv] = load_row8(dSt + ((2 * kv + (g >> 1)) * DK + 16 * m + li) * 16);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int kv = 0; kv < KV; ++kv) a = mma(dst[kv], fo[kv], a);
      a *= eta * br;
      const floatx4 k4 = ld4f(kl.x + tok * kl.kLd + 16 * m + 4 * g);
#pragma unroll
      for (int r = 0; r < 4; ++r) write += (double)k4[r] * (double)a[r];
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        if (ks < wave / 2) continue;
        a = mma(kl.transposed(m, ks, lane), load_frag<Op>(da_f + ks * kOpFrag, lane), a);
        a = mma(ql.transposed(m, ks, lane), load_frag<Op>(dp_f + ks * kOpFrag, lane), a);
      }
      settle(a);
      dk[i] += a;
#pragma unroll
      for (int r = 0; r < 4; ++r) dg -= (double)k4[r] * (double)a[r];
    }
    // the log-decay's gradient
    dg += __shfl_xor(dg, 16);
    dg += __shfl_xor(dg, 32);
    double ex = write + (double)last * hold;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) ex += __shfl_xor(ex, d);
    if (g == 0) dG[half][tok] = dg;
    if (lane == 0) extra[wave_id()] = ex;
    __syncthreads();
    if (wave_id() == 0) {
      double x = dG[0][lane] + dG[1][lane];
      if (lane == 63) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x += extra[i];
      }
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const double dn = __shfl_down(x, d);
        if (lane + d < 64) x += dn;
      }
      if (lane < n) {
        const float w = get(global_in<T>(p.w) + seq.row * p.sw.b + h * p.sw.h + (t0 + lane) * p.sw.t);
        put(global_out<T>(p.dw) + seq.row * p.sdw.b + h * p.sdw.h + (t0 + lane) * p.sdw.t,
            (float)(x * (double)gdr_gate_grad(w, p.gate, p.g_min)));
        const auto db = global_in<float>(p.ws_db) + blk * (DV / 16) * kGdrChunk + lane;
        float sum = 0.f;
#pragma unroll
        for (int c = 0; c < DV / 16; ++c) sum += db[c * kGdrChunk];
        put(global_out<T>(p.dbeta) + seq.row * p.sdb.b + h * p.sdb.h + (t0 + lane) * p.sdb.t, sum);
      }
    }
    __syncthreads();
  }

  const int tok = 16 * wave + (lane & 15), g = lane >> 4;
  if (tok < n) {
    const auto dqp = global_out<T>(p.dq) + seq.row * p.sdq.b + kh * p.sdq.h + (t0 + tok) * p.sdq.t + 4 * g;
    const auto dkp = global_out<T>(p.dk_) + seq.row * p.sdk.b + kh * p.sdk.h + (t0 + tok) * p.sdk.t + 4 * g;
#pragma unroll
    for (int i = 0; i < MH; ++i) {
      const int m = half * MH + i;
      store_row4(dqp + 16 * m, dq[i]);
      store_row4(dkp + 16 * m, dk[i]);
    }
  }
}

template <int DK, int DV>
hipError_t launch_one(const GdrParams& p, hipStream_t s) {
  const dim3 grid((unsigned)gdr_slots(p.B, p.T, p.n_seq, p.seq_start != nullptr), (unsigned)p.Hk);
  if (grid.x == 0) return hipSuccess;
  if (p.dtype == KDA_DTYPE_BF16) hipLaunchKernelGGL((gdr_grad_kernel<DK, DV>), grid, dim3(512), 0, s, p);
  else hipLaunchKernelGGL((gdr_grad_f32_kernel<DK, DV>), grid, dim3(512), 0, s, p);
  return hipGetLastError();
}

template <int DK>
hipError_t launch_dk(const GdrParams& p, hipStream_t s) {
  switch (p.dv) {
    case 32: return launch_one<DK, 32>(p, s);
    case 64: return launch_one<DK, 64>(p, s);
    default: return launch_one<DK, 128>(p, s);
  }
}

}  // namespace

hipError_t launch_gdr_grad(const GdrParams& p, hipStream_t s) {
  switch (p.dk) {
    case 32: return launch_dk<32>(p, s);
    case 64: return launch_dk<64>(p, s);
    default: return launch_dk<128>(p, s);
  }
}

}  // namespace kda
