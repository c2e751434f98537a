// ss_scan2_bwd_mfma.hip -- gradients of the multi-head scan for bf16, headdim 64 and 64 or 128
// states: the formulas and launches of ss_scan2_bwd.hip, with the products on the bf16 matrix
// instruction.
//
// x, B and C are bf16 and enter the products exactly.  float32 operands are split into bf16 parts
// that take a product each.  On the way to the float32 results (dA, ddt_bias, dh0) they are three,
// the whole value: w X and e^c gy that make the states, the states where they meet C and B, gy where
// it meets X.  (Two parts, 2^-17, left dA and ddt_bias 2.7e-6 and 3.2e-6 off at 4 x 4096 x 80 heads
// and dh0 2.4e-6; three 1.8e-7, 2.5e-7 and 1.2e-7, as plain float32.)  What ends in a bf16 result
// alone, whose half step is 2^-8, has two: M and K, the states where they meet gy and X (dC and dB),
// gy there and where it meets M (dx).  Products that have K down the rows of a tile read it with the
// LDS transpose read, so every tile is staged once.
//
// The states cross from the first launch to the second in float32, laid out as the first one holds
// them: [d_state / 16][channel][16 states].  The LDS has room for two 16-bit planes of each, so it
// holds the words' upper and lower halves, and the parts are formed as operands are read.
//
// What bounds it, at 4 x 4096 x 80 heads with 128 states: the states kernel 495 us, for 1.31 GB of
// states written and 0.62 fetched (3.9 TB/s; with two parts 248 without the stores, 494 without the
// products, so it is the stores: splitting each walk's states over two workgroups took 570,
// non-temporal stores the same 505, loads issued before the stores or another order of the chunks in
// memory 528).  The chunks kernel 865 us with the gate, for 2.02 GB fetched and 0.38 written: the
// VALU is busy for half of the time, the LDS for a quarter, the matrix units for a seventh, and with
// one workgroup of eight waves on a CU (160 KB of tiles) and three barriers a head they overlap
// little.  The third parts and the float64 sums are 190 us of it (675 before, the VALU busy for 0.37;
// the parts by dot products, in two thirds of the instructions, took the same).  Measured with two
// parts: sixteen waves of half the work the same (825 against 821 us), 32 x 32 tiles gained 3 %, M
// in one bf16 4 % (not kept: dx and dz would be off by more than their own rounding), a head's
// parameters fetched with its tiles 6 %.
#include "ss_head.h"
#include "ss_mfma.h"
#include "ss_scan2_bwd.h"

namespace ss {
namespace {

constexpr int kQ = kScan2BwdChunk;
constexpr int kP = 64;
constexpr int kPS = kP + 8;   // bf16 per row of the (step, channel) and (step, step) tiles: 36
                              // dwords, so that the four rows of a transpose read and the sixteen
                              // of a 16-byte read start in different banks

// The upper and lower halves of four words.
__device__ __forceinline__ uint2 highs(uint4 w) {
  return make_uint2(__builtin_amdgcn_perm(w.y, w.x, 0x07060302),
                    __builtin_amdgcn_perm(w.w, w.z, 0x07060302));
}
__device__ __forceinline__ uint2 lows(uint4 w) {
  return make_uint2(__builtin_amdgcn_perm(w.y, w.x, 0x05040100),
                    __builtin_amdgcn_perm(w.w, w.z, 0x05040100));
}
// (a, b) as three bf16 parts, which hold a float32 value whole.
__device__ __forceinline__ void split3(float a, float b, uint32_t& hi, uint32_t& mid,
                                       uint32_t& rest) {
  hi = pack_bf16(a, b);
  const float ra = a - lo_f(hi), rb = b - hi_f(hi);
  split2(ra, rb, mid, rest);
}
// From the upper (a bf16 part as they are) and lower halves of eight float32 values: what the upper
// ones leave as one more part, or as two, which are the rest of the value.
__device__ __forceinline__ void left2(uint32_t up, uint32_t low, float& a, float& b) {
  const uint32_t wa = __builtin_amdgcn_perm(up, low, 0x05040100);
  const uint32_t wb = __builtin_amdgcn_perm(up, low, 0x07060302);
  a = __uint_as_float(wa) - __uint_as_float(wa & 0xffff0000u);
  b = __uint_as_float(wb) - __uint_as_float(wb & 0xffff0000u);
}
__device__ __forceinline__ Op left(const Op& up, const Op& low) {
  Op mid;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float a, b;
    left2(up.w[j], low.w[j], a, b);
    mid.w[j] = pack_bf16(a, b);
  }
  return mid;
}
__device__ __forceinline__ void left(const Op& up, const Op& low, Op& mid, Op& rest) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float a, b;
    left2(up.w[j], low.w[j], a, b);
    split2(a, b, mid.w[j], rest.w[j]);
  }
}

// ------------------------------------------------------------------ the states

template <int N>
struct alignas(16) StateSmem {
  uint16_t in[kQ][N + 16];        // B or C, (step, state)
  uint16_t row[3][kQ][kPS];       // weighted x or gy in three parts, (step, channel)
  float weight[2][kQ];
};

// One workgroup per (batch row, head) and direction; wave w owns channels 16 w .. 16 w + 15.  (Three
// on a CU: left alone the compiler takes registers for two, 542 us for 496 at 4 x 4096 x 80 heads.)
template <int N, bool CUT>
__global__ __launch_bounds__(256, 3) void scan2_states_mfma_kernel(Scan2BwdArgs p) {
  constexpr int NT = N / 16;
  constexpr int UNITS = 2 * N, UPT = (UNITS + 255) / 256;  // (4-step, 8-state) pieces
  __shared__ StateSmem<N> sm;
  const int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, g4 = lane >> 4;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  // a walk that is cut: a workgroup has one chunk, from a state of 0
  const int64_t nc = p.n_chunks, units = p.batch * p.nheads * (CUT ? nc : 1);
  const bool back = blockIdx.x >= units;
  const int64_t unit = xcd_remap(back ? blockIdx.x - units : blockIdx.x, units);
  const int64_t bh = CUT ? unit / nc : unit, only = CUT ? unit - bh * nc : 0;
  const int64_t b = bh / p.nheads, h = bh - b * p.nheads, grp = h / (p.nheads / p.ngroups);
  const int64_t L = p.seqlen, H = p.nheads, gn = p.ngroups * N, hp = H * kP;
  const float A = p.A[h], bias = p.dt_bias ? p.dt_bias[h] : 0.0f;
  const uint16_t* in = static_cast<const uint16_t*>(back ? p.C : p.B) + b * L * gn + grp * N;
  const uint16_t* row = static_cast<const uint16_t*>(back ? p.dout : p.x) + b * L * hp + h * kP;
  const uint16_t* zrow =
      back && p.z ? static_cast<const uint16_t*>(p.z) + b * L * hp + h * kP : nullptr;
  const uint16_t* dtg = static_cast<const uint16_t*>(p.dt) + b * L * H + h;
  uint4* ws = reinterpret_cast<uint4*>(back ? p.lam : p.states) + bh * nc * (N * kP / 4);
  const float* init = CUT ? nullptr : back ? p.dh_last : p.h0;
  const int rq = tid >> 4, rp = tid & 15;  // this thread's 4 steps x 4 channels of the rows

  uint2 xr[4], zr[4];
  uint4 ir[UPT][4];
  uint16_t dtr = 0;
  auto fetch = [&](int64_t ch) {
    const int64_t t0 = ch * kQ, left = L - t0;
    const int nv = static_cast<int>(left < kQ ? left : kQ);
    dtr = lane < nv ? dtg[(t0 + lane) * H] : 0;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int t = 4 * rq + r;
      const int64_t o = (t0 + t) * hp + 4 * rp;
      xr[r] = t < nv ? *reinterpret_cast<const uint2*>(row + o) : make_uint2(0, 0);
      if (zrow) zr[r] = t < nv ? *reinterpret_cast<const uint2*>(zrow + o) : make_uint2(0, 0);
    }
#pragma unroll
    for (int k = 0; k < UPT; ++k) {
      const int u = tid + 256 * k, tq = u / (N / 8), nb = u % (N / 8);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int t = 4 * tq + r;
        ir[k][r] = u < UNITS && t < nv
                       ? *reinterpret_cast<const uint4*>(in + (t0 + t) * gn + 8 * nb)
                       : make_uint4(0, 0, 0, 0);
      }
    }
  };
  // w_s = dt e^{c_end - c_s} forward, e^{c_t} backward; the same bits from every wave
  float decay = 1.0f;
  auto weigh = [&](int64_t ch, int buf) {
    const Step s = step_of(BF16::widen(dtr), ch * kQ + lane < L, bias, A, p.softplus);
    decay = s.end;
    sm.weight[buf][lane] = back ? s.before : s.after * s.dt;
  };

  f32x4 S[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int r = 0; r < 4; ++r)
      S[nt][r] = init ? init[(bh * N + 16 * nt + 4 * g4 + r) * kP + 16 * wv + l16] : 0.0f;

  const int64_t chunks = CUT ? 1 : nc, first = CUT ? only : back ? nc - 1 : 0;
  fetch(first);
  weigh(first, 0);
  for (int64_t k = 0; k < chunks; ++k) {
    const int64_t ch = back ? first - k : first + k;
    __syncthreads();  // the previous chunk's tiles have been read, this one's weights are there
#pragma unroll
    for (int u8 = 0; u8 < UPT; ++u8) {
      const int u = tid + 256 * u8, tq = u / (N / 8), nb = u % (N / 8);
      if (UNITS % 256 == 0 || u < UNITS) {
#pragma unroll
        for (int r = 0; r < 4; ++r)
          *reinterpret_cast<uint4*>(&sm.in[4 * tq + r][8 * nb]) = ir[u8][r];
      }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const float w = sm.weight[k & 1][4 * rq + r];
      float v[4] = {lo_f(xr[r].x), hi_f(xr[r].x), lo_f(xr[r].y), hi_f(xr[r].y)};
      if (zrow) {
        const float z[4] = {lo_f(zr[r].x), hi_f(zr[r].x), lo_f(zr[r].y), hi_f(zr[r].y)};
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] *= z[j] * sigmoid_f(z[j]);
      }
      uint2 part[3];
      split3(v[0] * w, v[1] * w, part[0].x, part[1].x, part[2].x);
      split3(v[2] * w, v[3] * w, part[0].y, part[1].y, part[2].y);
#pragma unroll
      for (int q = 0; q < 3; ++q)
        *reinterpret_cast<uint2*>(&sm.row[q][4 * rq + r][4 * rp]) = part[q];
    }
    // the state before the chunk leaves before the next loads are issued, which would be waited
    // for together with it
    uint4* out = ws + ch * (N * kP / 4) + (16 * wv + l16) * 4 + g4;
    if (!CUT) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) out[nt * kP * 4] = __builtin_bit_cast(uint4, S[nt]);
    }
    const float d = decay;
    const bool more = k + 1 < chunks;
    const int64_t next = back ? ch - 1 : ch + 1;
    if (more) fetch(next);
    __syncthreads();
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) S[nt] *= d;
#pragma unroll
    for (int kb = 0; kb < kQ; kb += 32) {
      Op w[3];
#pragma unroll
      for (int q = 0; q < 3; ++q) w[q] = op_down(&sm.row[q][0][0], kPS, kb, 16 * wv, l16, g4);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const Op a = op_down(&sm.in[0][0], N + 16, kb, 16 * nt, l16, g4);
#pragma unroll
        for (int q = 0; q < 3; ++q) S[nt] = mfma(a, w[q], S[nt]);
      }
    }
    if (more) weigh(next, (k + 1) & 1);
    lds_reads_done();
  }
  if (CUT) {  // the chunk's own part
    uint4* out = ws + only * (N * kP / 4) + (16 * wv + l16) * 4 + g4;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) out[nt * kP * 4] = __builtin_bit_cast(uint4, S[nt]);
    if (tid == 0) p.decay[((back ? p.batch : 0) * H + bh) * nc + only] = decay;
  } else if (back && p.dh0) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        p.dh0[(bh * N + 16 * nt + 4 * g4 + r) * kP + 16 * wv + l16] = S[nt][r];
  }
}

// ------------------------------------------------------------------ the chunks

constexpr int kThreads = 512;  // eight waves, one workgroup on a CU

template <int N>
struct alignas(16) ChunkSmem {
  uint16_t b[kQ][N + 8], c[kQ][N + 8];           // B and C, (step, state)
  // S_in and lam_out, (channel, state): upper and lower halves
  uint16_t shi[kP][N + 8], slo[kP][N + 8];
  uint16_t lhi[kP][N + 8], llo[kP][N + 8];
  uint16_t x[kQ][kPS];                           // (step, channel)
  uint16_t ghi[kQ][kPS], glo[kQ][kPS];           // gy in parts
  uint16_t grest[kQ][kP];                        // (8-channel pieces at piece ^ (step & 7))
  uint16_t mhi[kQ][kPS], mlo[kQ][kPS];           // M dt_s, (t, s); at the end K
  float dt[kQ], c_hi[kQ], c_lo[kQ], before[kQ], after[kQ];
  // sums for dl and ddt: E / dt over t and E over s of each causal tile (strictly below the diagonal),
  // q, p / dt
  double ecol[10][16], erow[10][16];
  float near[2][kQ], far[2][kQ];
  float over[kThreads / 64], gx[kThreads / 64];  // <S_in, lam_out>, gy . x, by wave
  // the diagonal of W M, in the 16 bytes behind a row of x that keep the banks apart
  __device__ __forceinline__ float& ediag(int t) { return *reinterpret_cast<float*>(&x[t][kP]); }
};

// 32 x 32 tiles: the operand's rows (or columns) are 32 of the tile, lane % 32 each, K = k0 + 8
// (lane / 32) + 0..7; the result has column lane % 32, and in element 4 q + r row 8 q +
// 4 (lane / 32) + r.  Half the operand bytes of four 16 x 16 tiles per product.
using f32x16 = float __attribute__((ext_vector_type(16)));
__device__ __forceinline__ f32x16 mfma32(const Op& a, const Op& b, f32x16 c) {
  using u4 = uint32_t __attribute__((ext_vector_type(4)));
  const u4 av = {a.w[0], a.w[1], a.w[2], a.w[3]};
  const u4 bv = {b.w[0], b.w[1], b.w[2], b.w[3]};
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, av),
                                                 __builtin_bit_cast(bf16x8, bv), c, 0, 0, 0);
}
__device__ __forceinline__ Op along32(const uint16_t* tile, int stride, int r0, int k0, int lane) {
  const uint4 v = *reinterpret_cast<const uint4*>(tile + (r0 + (lane & 31)) * stride + k0 +
                                                  8 * (lane >> 5));
  return Op{{v.x, v.y, v.z, v.w}};
}
__device__ __forceinline__ Op down32(const uint16_t* tile, int stride, int k0, int c0, int lane) {
  const int k = k0 + 8 * (lane >> 5), c = c0 + (lane & 16), l16 = lane & 15;
  const uint2 k03 = tr_read4(tile, stride, k, c, l16), k47 = tr_read4(tile, stride, k + 4, c, l16);
  return Op{{k03.x, k03.y, k47.x, k47.y}};
}

template <int N, bool GATE>
__global__ __launch_bounds__(kThreads) void scan2_chunks_mfma_kernel(Scan2BwdArgs p) {
  constexpr int SK = N * kP / 4 / kThreads;  // 16-byte pieces of a state per thread
  constexpr int TPW = N / 64;                // 32 x 32 tiles of dB or dC per wave
  __shared__ ChunkSmem<N> sm;
  const int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, g4 = lane >> 4;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t nc = p.n_chunks, L = p.seqlen, H = p.nheads, hp = H * kP, gn = p.ngroups * N;
  int64_t w = blockIdx.x;
  const int64_t split = w % p.splits;
  w /= p.splits;
  const int64_t grp = w % p.ngroups;
  w /= p.ngroups;
  const int64_t ch = w % nc, b = w / nc, t0 = ch * kQ;
  const int rows = L - t0 < kQ ? static_cast<int>(L - t0) : kQ;
  const int64_t hg = H / p.ngroups;
  const int64_t h_beg = grp * hg + split * hg / p.splits,
                h_end = grp * hg + (split + 1) * hg / p.splits;

  // B and C of the chunk
  {
    const uint16_t* Bg = static_cast<const uint16_t*>(p.B) + (b * L + t0) * gn + grp * N;
    const uint16_t* Cg = static_cast<const uint16_t*>(p.C) + (b * L + t0) * gn + grp * N;
    for (int u = tid; u < kQ * N / 8; u += kThreads) {
      const int t = u / (N / 8), n = 8 * (u % (N / 8));
      uint4 bw = make_uint4(0, 0, 0, 0), cw = bw;
      if (t < rows) {
        bw = *reinterpret_cast<const uint4*>(Bg + t * gn + n);
        cw = *reinterpret_cast<const uint4*>(Cg + t * gn + n);
      }
      *reinterpret_cast<uint4*>(&sm.b[t][n]) = bw;
      *reinterpret_cast<uint4*>(&sm.c[t][n]) = cw;
    }
  }
  // the zeros above the diagonal are never written again
  {
    uint4* m = reinterpret_cast<uint4*>(&sm.mhi[0][0]);
    for (int i = tid; i < 2 * kQ * kPS * 2 / 16; i += kThreads) m[i] = make_uint4(0, 0, 0, 0);
  }
  __syncthreads();

  // The causal 16x16 tiles (s-tile ti <= t-tile tj), dealt to the waves in the order (0,0) (0,1)
  // (1,1) (0,2) ...: lane (l16, g4) holds steps s = 16 ti + 4 g4 + r and t = 16 tj + l16.
  int ti[2], tj[2];
  f32x4 G[2] = {}, K[2] = {};  // B C^T of them, and the sum of K over the heads
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int k = wv + 8 * i;
    tj[i] = (k >= 1) + (k >= 3) + (k >= 6);
    ti[i] = k - tj[i] * (tj[i] + 1) / 2;
    if (k < 10) {
#pragma unroll
      for (int kb = 0; kb < N; kb += 32)
        G[i] = mfma(op_along(&sm.b[0][0], N + 8, 16 * ti[i], kb, l16, g4),
                    op_along(&sm.c[0][0], N + 8, 16 * tj[i], kb, l16, g4), G[i]);
    }
  }
  const int mine = wv < 2 ? 2 : 1;
  // Waves 0 to 3 form Y and dC, waves 4 to 7 V and dB, transposed (rows: channels or states,
  // columns: steps): a tile of 32 channels and 32 steps each, and TPW tiles of 32 states.
  const int role = wv >> 2, ph = (wv >> 1) & 1, sh = wv & 1;
  const int nt = N == 128 ? wv & 3 : ph, j0 = N == 128 ? 0 : sh;
  const uint16_t* hi_t = role ? &sm.lhi[0][0] : &sm.shi[0][0];  // (channel, state)
  const uint16_t* lo_t = role ? &sm.llo[0][0] : &sm.slo[0][0];
  const uint16_t* bc_t = role ? &sm.b[0][0] : &sm.c[0][0];      // (step, state)
  const uint16_t* by_t = role ? &sm.x[0][0] : &sm.ghi[0][0];    // (step, channel)
  f32x16 dBC[TPW] = {};

  // A head's inputs on their way: 16-byte pieces of the states, 8 channels of one step of the rows
  uint4 sr[SK], lr[SK], xr, gr, zr;
  uint16_t dtr = 0;
  const int r8 = tid >> 3, c8 = (tid & 7) * 8;
  // (buffer resources: a row past the last step reads as 0, and an access costs one offset)
  const uint32_t row_bytes = static_cast<uint32_t>(hp * 2);
  const uint32_t tile_bytes = static_cast<uint32_t>(rows - 1) * row_bytes + kP * 2;
  const uint32_t row_off = r8 * row_bytes + c8 * 2;
  const uint32_t out_off = (32 * sh + (lane & 31)) * row_bytes + (32 * ph + 4 * (lane >> 5)) * 2;
  // (the head's parameters too: a load that is waited for at once would stand in every head's way)
  float An = 0.0f, Dn = 0.0f, bn = 0.0f;
  const uint32_t dt_off = lane * static_cast<uint32_t>(H * 2);
  const uint32_t dt_bytes = static_cast<uint32_t>((rows - 1) * H * 2) + 2;
  const rsrc_t ra = make_buf(p.A, static_cast<uint32_t>(H * 4));
  const rsrc_t rd = make_buf(p.D, p.D ? static_cast<uint32_t>(H * 4) : 0);
  const rsrc_t rb = make_buf(p.dt_bias, p.dt_bias ? static_cast<uint32_t>(H * 4) : 0);
  auto fetch = [&](int64_t h) {
    const int64_t o = (b * L + t0) * hp + h * kP;
    dtr = buf_load<uint16_t>(
        make_buf(static_cast<const uint16_t*>(p.dt) + (b * L + t0) * H + h, dt_bytes), dt_off);
    An = buf_load<float>(ra, static_cast<uint32_t>(h * 4));
    Dn = buf_load<float>(rd, static_cast<uint32_t>(h * 4));
    bn = buf_load<float>(rb, static_cast<uint32_t>(h * 4));
    xr = buf_load<uint4>(make_buf(static_cast<const uint16_t*>(p.x) + o, tile_bytes), row_off);
    gr = buf_load<uint4>(make_buf(static_cast<const uint16_t*>(p.dout) + o, tile_bytes), row_off);
    if (GATE)
      zr = buf_load<uint4>(make_buf(static_cast<const uint16_t*>(p.z) + o, tile_bytes), row_off);
    const int64_t at = ((b * H + h) * nc + ch) * (N * kP);
    const rsrc_t sp = make_buf(p.states + at, N * kP * 4), lp = make_buf(p.lam + at, N * kP * 4);
#pragma unroll
    for (int k = 0; k < SK; ++k) {
      sr[k] = __builtin_bit_cast(
          uint4, __builtin_amdgcn_raw_buffer_load_b128(sp, tid * 16, k * kThreads * 16, 0));
      lr[k] = __builtin_bit_cast(
          uint4, __builtin_amdgcn_raw_buffer_load_b128(lp, tid * 16, k * kThreads * 16, 0));
    }
  };

  // dl, ddt and the head's sums from what the products left (one wave)
  auto finish = [&](int64_t h, float A, const Step& st) {
    const float q = sm.near[0][lane] + sm.near[1][lane];
    const float f = sm.far[0][lane] + sm.far[1][lane];
    // the step's tiles: those of its row (as t), those of its column (as s)
    double col = 0.0, row = 0.0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (k <= g4) row += sm.erow[g4 * (g4 + 1) / 2 + k][l16];
      if (k >= g4) col += sm.ecol[k * (k + 1) / 2 + g4][l16];
    }
    const float xv = f + (static_cast<float>(col) + sm.ediag(lane));
    float ov = 0.0f, gx = 0.0f;
#pragma unroll
    for (int k = 0; k < kThreads / 64; ++k) {
      ov += sm.over[k];
      gx += sm.gx[k];
    }
    // inclusive sums in float64; what lies before a step is the sum less its own
    const double in = st.dt * col - row, ps = static_cast<double>(st.dt) * f;
    const double before = scan64(in + ps) - (in + ps);
    const double upto = scan64(q), since = last_lane(upto) - (upto - q);
    const float dl = static_cast<float>(before + since + static_cast<double>(st.end) * ov);
    float ddt = fmaf(A, dl, xv);
    ddt *= st.slope;
    if (lane < rows)
      static_cast<uint16_t*>(p.ddt)[(b * L + t0 + lane) * H + h] = BF16::from_float(ddt);
    else
      ddt = 0.0f;
    const float sa = sum64(st.dt * dl), sb = sum64(ddt);
    if (lane == 0) {
      float* line = p.head_part + (b * nc + ch) * 3 * H + h;
      line[0] = sa;
      line[H] = gx;
      line[2 * H] = sb;
    }
  };

  fetch(h_beg);
  float A = 0.0f;
  Step st{};
  const int lane0 = lane;
  for (int64_t h = h_beg; h < h_end; ++h) {
    // (hides that the lane's places in the tiles stay the same from head to head: the compiler
    // would keep some sixty addresses in registers, and spill; a spilled value's reload waits for
    // the loads of the next head, which were issued before it)
    int lane = lane0;
    asm volatile("" : "+v"(lane));
    const int l16 = lane & 15, g4 = lane >> 4, l32 = lane & 31, hi32 = lane >> 5;
    __syncthreads();  // the previous head's tiles have been read, its sums are there
    if (wv == 7 && h > h_beg) finish(h - 1, A, st);
    const float Dh = Dn;
    A = An;
    if (wv == 0 || wv == 7)
      st = step_of(BF16::widen(dtr), lane < rows, bn, A, p.softplus);
    if (wv == 0) {
      sm.dt[lane] = st.dt;
      sm.c_hi[lane] = st.c_hi;
      sm.c_lo[lane] = st.c_lo;
      sm.before[lane] = st.before;
      sm.after[lane] = st.after;
    }
    float over = 0.0f, gx = 0.0f;
#pragma unroll
    for (int k = 0; k < SK; ++k) {
      const int u = tid + kThreads * k, ch16 = (u >> 2) & (kP - 1), n = 16 * (u >> 8) + 4 * (u & 3);
      *reinterpret_cast<uint2*>(&sm.shi[ch16][n]) = highs(sr[k]);
      *reinterpret_cast<uint2*>(&sm.slo[ch16][n]) = lows(sr[k]);
      *reinterpret_cast<uint2*>(&sm.lhi[ch16][n]) = highs(lr[k]);
      *reinterpret_cast<uint2*>(&sm.llo[ch16][n]) = lows(lr[k]);
      const f32x4 a = __builtin_bit_cast(f32x4, sr[k]), c = __builtin_bit_cast(f32x4, lr[k]);
#pragma unroll
      for (int j = 0; j < 4; ++j) over = fmaf(a[j], c[j], over);
    }
    *reinterpret_cast<uint4*>(&sm.x[r8][c8]) = xr;
    {
      const uint32_t gw[4] = {gr.x, gr.y, gr.z, gr.w}, zw[4] = {zr.x, zr.y, zr.z, zr.w};
      uint32_t hi[4], lo[4], rest[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float a = lo_f(gw[j]), c = hi_f(gw[j]);
        if (GATE) {
          const float za = lo_f(zw[j]), zc = hi_f(zw[j]);
          a *= za * sigmoid_f(za);
          c *= zc * sigmoid_f(zc);
        }
        const uint32_t xw = j == 0 ? xr.x : j == 1 ? xr.y : j == 2 ? xr.z : xr.w;
        gx = fmaf(a, lo_f(xw), fmaf(c, hi_f(xw), gx));
        split3(a, c, hi[j], lo[j], rest[j]);
      }
      *reinterpret_cast<uint4*>(&sm.ghi[r8][c8]) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
      *reinterpret_cast<uint4*>(&sm.glo[r8][c8]) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
      if (GATE)
        *reinterpret_cast<uint4*>(&sm.grest[r8][c8 ^ (r8 & 7) * 8]) =
            make_uint4(rest[0], rest[1], rest[2], rest[3]);
    }
    __syncthreads();  // the tiles are there
    // z and dout again for the epilogue, in its layout (they lie in the caches); then the next head
    uint2 ze[4], ge[4];
    const int64_t tile0 = (b * L + t0) * hp + h * kP;
    if (GATE && !role) {
      const rsrc_t rz = make_buf(static_cast<const uint16_t*>(p.z) + tile0, tile_bytes);
      const rsrc_t rg = make_buf(static_cast<const uint16_t*>(p.dout) + tile0, tile_bytes);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        ze[q] = buf_load<uint2>(rz, out_off + 16 * q);
        ge[q] = buf_load<uint2>(rg, out_off + 16 * q);
      }
    }
    __builtin_amdgcn_sched_barrier(0);  // in this order: loads are waited for in theirs
    // (the last head fetches itself again: the compiler counts loads, and takes what may not have
    // been issued for what it waits for)
    fetch(h + 1 < h_end ? h + 1 : h);
    __builtin_amdgcn_sched_barrier(0);

    // ---- W = X gy^T over the causal tiles; M dt to LDS, K into its sum, the sums of E
    over = sum64(over);
    gx = sum64(gx);
    if (lane == 0) {
      sm.over[wv] = over;
      sm.gx[wv] = gx;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (i >= mine) continue;
      f32x4 W = {};
#pragma unroll
      for (int kb = 0; kb < kP; kb += 32) {
        const Op a = op_along(&sm.x[0][0], kPS, 16 * ti[i], kb, l16, g4);
        W = mfma(a, op_along(&sm.ghi[0][0], kPS, 16 * tj[i], kb, l16, g4), W);
        W = mfma(a, op_along(&sm.glo[0][0], kPS, 16 * tj[i], kb, l16, g4), W);
        if (GATE) {
          const uint4 r = *reinterpret_cast<const uint4*>(
              &sm.grest[16 * tj[i] + l16][(kb + 8 * g4) ^ (l16 & 7) * 8]);
          W = mfma(a, Op{{r.x, r.y, r.z, r.w}}, W);
        }
      }
      const int t = 16 * tj[i] + l16, s0 = 16 * ti[i] + 4 * g4;
      const float cth = sm.c_hi[t], ctl = sm.c_lo[t];
      const float4 csh = *reinterpret_cast<const float4*>(&sm.c_hi[s0]);
      const float4 csl = *reinterpret_cast<const float4*>(&sm.c_lo[s0]);
      const float4 dt4 = *reinterpret_cast<const float4*>(&sm.dt[s0]);
      const float ch[4] = {csh.x, csh.y, csh.z, csh.w}, cl[4] = {csl.x, csl.y, csl.z, csl.w};
      const float dts[4] = {dt4.x, dt4.y, dt4.z, dt4.w};
      float m[4], e[4];
      double row = 0.0, col[4];
      const bool diag = ti[i] == tj[i];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float seg = exp2_diff(cth, ctl, ch[r], cl[r]);
        const bool in = !diag || s0 + r <= t;
        m[r] = in ? G[i][r] * seg : 0.0f;
        e[r] = in ? W[r] * m[r] : 0.0f;
        K[i][r] += in ? W[r] * seg * dts[r] : 0.0f;
        m[r] *= dts[r];
      }
      uint2 h2, l2;
      split2(m[0], m[1], h2.x, l2.x);
      split2(m[2], m[3], h2.y, l2.y);
      *reinterpret_cast<uint2*>(&sm.mhi[t][s0]) = h2;
      *reinterpret_cast<uint2*>(&sm.mlo[t][s0]) = l2;
      if (diag) {  // the diagonal itself apart
        float ed = 0.0f;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const bool on = s0 + r == t;
          ed += on ? e[r] : 0.0f;
          e[r] = on ? 0.0f : e[r];
        }
        ed = sum_rows(ed);
        if (g4 == 0) sm.ediag(t) = ed;
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        row = fma(static_cast<double>(e[r]), static_cast<double>(dts[r]), row);
        col[r] = sum16(static_cast<double>(e[r]));
      }
      row = sum_rows(row);
      if (g4 == 0) sm.erow[wv + 8 * i][l16] = row;
      if (l16 == 0) {
#pragma unroll
        for (int r = 0; r < 4; ++r) sm.ecol[wv + 8 * i][4 * g4 + r] = col[r];
      }
    }

    // ---- S_in^T C^T or lam_out^T B^T
    f32x16 Y = {};
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll 2
    for (int kb = 0; kb < N; kb += 16) {
      const Op to = along32(bc_t, N + 8, 32 * sh, kb, lane);
      const Op up = along32(hi_t, N + 8, 32 * ph, kb, lane);
      Op mid, rest;
      left(up, along32(lo_t, N + 8, 32 * ph, kb, lane), mid, rest);
      Y = mfma32(up, to, Y);
      Y = mfma32(mid, to, Y);
      Y = mfma32(rest, to, Y);
    }
    // ---- S_in gy^T or lam_out X^T, scaled by their steps into dC or dB
    {
      f32x16 T[TPW] = {};
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll 2
      for (int kb = 0; kb < kP; kb += 16) {
        const Op ah = down32(hi_t, N + 8, kb, 32 * nt, lane);
        const Op al = left(ah, down32(lo_t, N + 8, kb, 32 * nt, lane));
#pragma unroll
        for (int j = 0; j < TPW; ++j) {
          const Op to = along32(by_t, kPS, 32 * (j0 + j), kb, lane);
          T[j] = mfma32(ah, to, T[j]);
          T[j] = mfma32(al, to, T[j]);
          if (!role) T[j] = mfma32(ah, along32(&sm.glo[0][0], kPS, 32 * (j0 + j), kb, lane), T[j]);
        }
      }
#pragma unroll
      for (int j = 0; j < TPW; ++j) {
        const int t = 32 * (j0 + j) + l32;
        const float by = role ? sm.after[t] * sm.dt[t] : sm.before[t];
#pragma unroll
        for (int r = 0; r < 16; ++r) dBC[j][r] = fmaf(by, T[j][r], dBC[j][r]);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    __syncthreads();  // M is there

    // ---- the carried parts scaled and summed, then the chunk's own: X^T (M dt)^T over s <= t, or
    // gy^T (M dt) over t >= s
    const int t = 32 * sh + l32, c0 = 32 * ph + 4 * hi32;
    const float dts = sm.dt[t], by = role ? sm.after[t] : sm.before[t];
    float part = 0.0f;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      float v[4];
      if (role) {
        const uint2 xw = *reinterpret_cast<const uint2*>(&sm.x[t][c0 + 8 * q]);
        v[0] = lo_f(xw.x), v[1] = hi_f(xw.x), v[2] = lo_f(xw.y), v[3] = hi_f(xw.y);
      } else {
        const uint2 gh = *reinterpret_cast<const uint2*>(&sm.ghi[t][c0 + 8 * q]);
        const uint2 gl = *reinterpret_cast<const uint2*>(&sm.glo[t][c0 + 8 * q]);
        v[0] = lo_f(gh.x) + lo_f(gl.x), v[1] = hi_f(gh.x) + hi_f(gl.x);
        v[2] = lo_f(gh.y) + lo_f(gl.y), v[3] = hi_f(gh.y) + hi_f(gl.y);
        if (GATE) {
          const uint2 gr = *reinterpret_cast<const uint2*>(
              &sm.grest[t][(c0 + 8 * q) ^ (t & 7) * 8]);
          v[0] += lo_f(gr.x), v[1] += hi_f(gr.x), v[2] += lo_f(gr.y), v[3] += hi_f(gr.y);
        }
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        Y[4 * q + r] *= by;
        part = fmaf(v[r], Y[4 * q + r], part);
        if (role) Y[4 * q + r] *= dts;
      }
    }
    part = sum_halves(part);
    if (hi32 == 0) (role ? sm.far : sm.near)[ph][t] = part;
    if (role) {
      for (int kb = 32 * sh; kb < kQ; kb += 16) {
        const Op ga = down32(&sm.ghi[0][0], kPS, kb, 32 * ph, lane);
        const Op gb = down32(&sm.glo[0][0], kPS, kb, 32 * ph, lane);
        const Op ma = down32(&sm.mhi[0][0], kPS, kb, 32 * sh, lane);
        const Op mb = down32(&sm.mlo[0][0], kPS, kb, 32 * sh, lane);
        Y = mfma32(ga, ma, Y);
        Y = mfma32(gb, ma, Y);
        Y = mfma32(ga, mb, Y);
      }
      const rsrc_t rx = make_buf(static_cast<uint16_t*>(p.dx) + tile0, tile_bytes);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint2 gh = *reinterpret_cast<const uint2*>(&sm.ghi[t][c0 + 8 * q]);
        const uint2 gl = *reinterpret_cast<const uint2*>(&sm.glo[t][c0 + 8 * q]);
        const float gy[4] = {lo_f(gh.x) + lo_f(gl.x), hi_f(gh.x) + hi_f(gl.x),
                             lo_f(gh.y) + lo_f(gl.y), hi_f(gh.y) + hi_f(gl.y)};
        float dx[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) dx[r] = fmaf(Dh, gy[r], Y[4 * q + r]);
        store8(make_uint2(pack_bf16(dx[0], dx[1]), pack_bf16(dx[2], dx[3])), rx, out_off + 16 * q);
      }
    } else if (GATE) {
      for (int kb = 0; kb < 32 * (sh + 1); kb += 16) {
        const Op xo = down32(&sm.x[0][0], kPS, kb, 32 * ph, lane);
        Y = mfma32(xo, along32(&sm.mhi[0][0], kPS, 32 * sh, kb, lane), Y);
        Y = mfma32(xo, along32(&sm.mlo[0][0], kPS, 32 * sh, kb, lane), Y);
      }
      const rsrc_t rz = make_buf(static_cast<uint16_t*>(p.dz) + tile0, tile_bytes);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint2 xw = *reinterpret_cast<const uint2*>(&sm.x[t][c0 + 8 * q]);
        const float x[4] = {lo_f(xw.x), hi_f(xw.x), lo_f(xw.y), hi_f(xw.y)};
        const float z[4] = {lo_f(ze[q].x), hi_f(ze[q].x), lo_f(ze[q].y), hi_f(ze[q].y)};
        const float go[4] = {lo_f(ge[q].x), hi_f(ge[q].x), lo_f(ge[q].y), hi_f(ge[q].y)};
        float dz[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float sg = sigmoid_f(z[r]);
          dz[r] = go[r] * fmaf(Dh, x[r], Y[4 * q + r]) * (sg * fmaf(z[r], 1.0f - sg, 1.0f));
        }
        store8(make_uint2(pack_bf16(dz[0], dz[1]), pack_bf16(dz[2], dz[3])), rz, out_off + 16 * q);
      }
    }
    lds_reads_done();
  }
  __syncthreads();
  if (wv == 7) finish(h_end - 1, A, st);

  // ---- dC^T += B^T K^T, dB^T += C^T K, K (t, s) in M's place
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (i >= mine) continue;
    const int t = 16 * tj[i] + l16, s0 = 16 * ti[i] + 4 * g4;
    uint2 h2, l2;
    split2(K[i][0], K[i][1], h2.x, l2.x);
    split2(K[i][2], K[i][3], h2.y, l2.y);
    *reinterpret_cast<uint2*>(&sm.mhi[t][s0]) = h2;
    *reinterpret_cast<uint2*>(&sm.mlo[t][s0]) = l2;
  }
  __syncthreads();
  const uint16_t* kt = role ? &sm.c[0][0] : &sm.b[0][0];
#pragma unroll
  for (int kb = 0; kb < kQ; kb += 16) {
    const Op a = down32(kt, N + 8, kb, 32 * nt, lane);
#pragma unroll
    for (int j = 0; j < TPW; ++j) {
      const int c = 32 * (j0 + j);
      dBC[j] = mfma32(a, role ? down32(&sm.mhi[0][0], kPS, kb, c, lane)
                              : along32(&sm.mhi[0][0], kPS, c, kb, lane), dBC[j]);
      dBC[j] = mfma32(a, role ? down32(&sm.mlo[0][0], kPS, kb, c, lane)
                              : along32(&sm.mlo[0][0], kPS, c, kb, lane), dBC[j]);
    }
  }
#pragma unroll
  for (int j = 0; j < TPW; ++j) {
    const int t = 32 * (j0 + j) + (lane & 31);
    if (t >= rows) continue;
    const int64_t o =
        ((b * L + t0 + t) * p.ngroups + grp) * N + 32 * nt + 4 * (lane >> 5);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float v[4] = {dBC[j][4 * q], dBC[j][4 * q + 1], dBC[j][4 * q + 2], dBC[j][4 * q + 3]};
      if (p.splits == 1) {
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(role ? p.dB : p.dC) + o + 8 * q) =
            make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
      } else {
        const int64_t all = p.batch * L * gn;
        *reinterpret_cast<float4*>(p.bc_part + split * 2 * all + (role ? 0 : all) + o + 8 * q) =
            make_float4(v[0], v[1], v[2], v[3]);
      }
    }
  }
}

template <int N>
hipError_t launch_n(const Scan2BwdArgs& a, hipStream_t stream) {
  const int64_t walks = 2 * a.batch * a.nheads;
  if (a.cut) {
    hipLaunchKernelGGL((scan2_states_mfma_kernel<N, true>),
                       dim3(static_cast<unsigned>(walks * a.n_chunks)), dim3(256), 0, stream, a);
    const hipError_t e = launch_scan2_join(a, true, stream);
    if (e != hipSuccess) return e;
  } else {
    hipLaunchKernelGGL((scan2_states_mfma_kernel<N, false>), dim3(static_cast<unsigned>(walks)),
                       dim3(256), 0, stream, a);
  }
  const dim3 grid(static_cast<unsigned>(a.batch * a.n_chunks * a.ngroups * a.splits));
  if (a.z)
    hipLaunchKernelGGL((scan2_chunks_mfma_kernel<N, true>), grid, dim3(kThreads), 0, stream, a);
  else
    hipLaunchKernelGGL((scan2_chunks_mfma_kernel<N, false>), grid, dim3(kThreads), 0, stream, a);
  return hipGetLastError();
}

}  // namespace

// (a chunk's rows are addressed with 32-bit byte offsets)
bool scan2_bwd_mfma_supported(const Scan2BwdArgs& a, bool bf16) {
  const uintptr_t al =
      reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.z) |
      reinterpret_cast<uintptr_t>(a.B) | reinterpret_cast<uintptr_t>(a.C) |
      reinterpret_cast<uintptr_t>(a.dout) | reinterpret_cast<uintptr_t>(a.dx) |
      reinterpret_cast<uintptr_t>(a.dz) | reinterpret_cast<uintptr_t>(a.dB) |
      reinterpret_cast<uintptr_t>(a.dC);
  return bf16 && a.headdim == kP && (a.d_state == 64 || a.d_state == 128) && (al & 15) == 0 &&
         kQ * a.nheads * kP * 2 < (int64_t(1) << 31);  // covers the rows of dt and the heads' A
}

hipError_t launch_scan2_bwd_mfma(const Scan2BwdArgs& a, hipStream_t stream) {
  return a.d_state == 64 ? launch_n<64>(a, stream) : launch_n<128>(a, stream);
}

}  // namespace ss
