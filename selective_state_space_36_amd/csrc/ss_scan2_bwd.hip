// ss_scan2_bwd.hip -- gradients of the multi-head scan (ss_scan2.hip states the recurrence), in its
// chunked dual form on the matrix cores.
//
// For a head let S_t be the states (d_state x headdim), y' = C_t S_t, gy_t = dout_t silu(z_t), and
// lam_t = dL/dS_t = C_t gy_t^T + a_{t+1} lam_{t+1}.  Inside a chunk of Q steps, with c_t the sum of
// log a up to t, S_in the state before the chunk and lam_out the adjoint of the state behind it:
//
//     seg[t,s] = e^{c_t - c_s} (s <= t),   M = (C B^T) o seg,   K = (gy X^T) o seg o dt_s
//     Y'  = M dt X + e^{c} C S_in          V_s = lam_s^T B_s:  V = M^T gy + e^{c_end - c} B lam_out
//     dX  = D gy + dt V                    dz = dout (Y' + D X) silu'(z)
//     dC  = K B + e^{c} gy S_in^T          dB = K^T C + dt e^{c_end - c} X lam_out^T
//     dl_t = d / d log a_t = <lam_t, a_t S_{t-1}>: all that flows from before t to t or later,
//          = sum_{s < t <= t'} E[t',s] + sum_{t' >= t} q_{t'} + sum_{s < t} p_s + e^{c_end} <lam_out, S_in>
//       with E = K o M without its diagonal, q_t = gy_t . e^{c_t} C_t S_in and
//       p_s = dt_s x_s . e^{c_end - c_s} B_s lam_out.  (The difference of y' gy and dt x V summed
//       from the end gives the same and cancels; here only the sum of E is a difference, of column
//       sums and row sums up to t.  Those are formed in float64: rounded to float32 their roundings
//       would walk through the chunk and stay where E itself has ended, which made dA up to 1.1e-5
//       off at fast decays, 3 x 777, 6 heads of 48 x 40; 1.1e-6 so, and plain float32 2.5e-6.)
//     ddt = (A dl + x . V) softplus',   dA = sum dt dl,   dD = sum gy x
//
// Three launches.  states: one workgroup per (batch row, head, 64 channels) walks the chunks and
// writes S_in, others walk them backwards and write lam_out (their state in registers); for few
// heads there is one per chunk instead, from a state of 0, and a fourth launch joins them.  chunks:
// one workgroup per (batch row, chunk, run of heads of one group) forms everything else, and adds
// K, e^c gy S_in^T and w X lam_out^T over its heads in registers, so that C B^T is formed once for
// them and dB and dC leave once.  sums: dB and dC over the runs, and the per-chunk sums of dA, dD
// and ddt_bias, in a fixed order.
//
// All products run as v_mfma_f32_16x16x4_f32 here: operands of every type and size, exact in
// float32.  Sizes that are not multiples of the tiles are filled with zeros.  What bounds it: at
// 4 x 4096, 80 heads of 64 x 128 float32 the chunks take 2340 us and the states 1080, three times
// what the chunks' products, 1.1e11 operations, take at the rate of a large float32 product (147
// TFLOP/s).  dC and dB of every block of 64 states stay in registers through the heads, and the
// chunks kernel spills: 19, 41, 57 and 77 of its 256 for one to four blocks, stored and reloaded in
// every head, with one workgroup on a CU (125 KB of tiles) and its barriers beside them.  4 x 2048, 40
// heads of 64 x 256 bf16: chunks 995, states 660.  For few heads it is latency: 3 x 777, 6 heads of 48
// x 40 float32, 36 walks of 13 chunks, states 10 us and their join 5 (37 walked whole), chunks 27.
#include "ss_head.h"
#include "ss_mfma.h"
#include "ss_octs.h"
#include "ss_rows.h"
#include "ss_scan2_bwd.h"

namespace ss {
namespace {

constexpr int kQ = kScan2BwdChunk;   // steps of a chunk, and the side of every tile
constexpr int kPitch = kQ + 4;       // floats per tile row: 16 rows start 4 banks apart, so 16-byte
                                     // reads of a column of rows, and 4-byte reads of rows four
                                     // apart, are free of bank conflicts

// The operand of four MFMA steps: lane (l16, g4) holds row (or column) l16 and, at step j, the
// inner index 4 g4 + j of the block of 16.
struct Frag {
  float v[4];
};
// Inner index along the tile's rows ...
__device__ __forceinline__ Frag along(const float* tile, int r0, int k0, int l16, int g4) {
  const float4 q = *reinterpret_cast<const float4*>(tile + (r0 + l16) * kPitch + k0 + 4 * g4);
  return Frag{{q.x, q.y, q.z, q.w}};
}
// ... and down its columns.
__device__ __forceinline__ Frag down(const float* tile, int k0, int c0, int l16, int g4) {
  Frag f;
#pragma unroll
  for (int j = 0; j < 4; ++j) f.v[j] = tile[(k0 + 4 * g4 + j) * kPitch + c0 + l16];
  return f;
}
__device__ __forceinline__ Frag operator*(Frag f, float s) {
#pragma unroll
  for (int j = 0; j < 4; ++j) f.v[j] *= s;
  return f;
}
// Scaled by the inner index.
__device__ __forceinline__ Frag scaled(Frag f, const float* by, int k0, int g4) {
  const float4 q = *reinterpret_cast<const float4*>(by + k0 + 4 * g4);
  f.v[0] *= q.x;
  f.v[1] *= q.y;
  f.v[2] *= q.z;
  f.v[3] *= q.w;
  return f;
}
__device__ __forceinline__ f32x4 mac(const Frag& a, const Frag& b, f32x4 c) {
#pragma unroll
  for (int j = 0; j < 4; ++j) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.v[j], b.v[j], c, 0, 0, 0);
  return c;
}

// The chunk's steps, one per lane.
template <class IO>
__device__ __forceinline__ Step steps(const Scan2BwdArgs& p, int64_t b, int64_t h, int64_t t0,
                                      int lane) {
  const bool in = t0 + lane < p.seqlen;
  const float dt = in ? IO::widen(static_cast<const typename IO::elem*>(
                            p.dt)[(b * p.seqlen + t0 + lane) * p.nheads + h])
                      : 0.0f;
  return step_of(dt, in, p.dt_bias ? p.dt_bias[h] : 0.0f, p.A[h], p.softplus);
}

// A thread's eight values of a 64 x 64 tile: row tid / 8, columns 8 (tid % 8).. of the `rows` x
// `cols` that are there (the rest 0).
template <class IO>
__device__ __forceinline__ void tile8(const typename IO::elem* base, int64_t pitch, int rows,
                                      int cols, int r, int c, float (&v)[8]) {
  load8<IO>(base + r * pitch + c, r < rows ? cols - c : 0, v);
}
__device__ __forceinline__ void put8(float* tile, int r, int c, const float (&v)[8]) {
  float4* q = reinterpret_cast<float4*>(tile + r * kPitch + c);
  q[0] = make_float4(v[0], v[1], v[2], v[3]);
  q[1] = make_float4(v[4], v[5], v[6], v[7]);
}

// ------------------------------------------------------------------ the states

template <int NB>
struct alignas(16) StateSmem {
  float in[NB][kQ * kPitch];  // B or C, (step, state)
  float row[kQ * kPitch];     // weighted x or gy, (step, channel)
  float weight[kQ];
};

// NB: 64-state blocks.  Workgroups 0 .. n - 1 walk forward (S_in), the others backward (lam_out);
// wave w holds channels 16 (w % 4).. and every other state tile from w / 4 on.  The next chunk is
// asked for before this one's products.
template <class IO, int NB>
__global__ __launch_bounds__(512) void scan2_states_kernel(Scan2BwdArgs p) {
  using E = typename IO::elem;
  constexpr int NT = 2 * NB;
  __shared__ StateSmem<NB> sm;
  const int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, g4 = lane >> 4;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6), pw = wv & 3, nw = wv >> 2;
  const int64_t half = gridDim.x / 2;
  const bool back = blockIdx.x >= half;
  int64_t w = back ? blockIdx.x - half : blockIdx.x;
  // a walk that is cut: this workgroup has one chunk, from a state of 0
  const int64_t only = p.cut ? w % p.n_chunks : 0;
  if (p.cut) w /= p.n_chunks;
  const int64_t pb = w % p.n_pblk;
  w /= p.n_pblk;
  const int64_t b = w / p.nheads, h = w - b * p.nheads, grp = h / (p.nheads / p.ngroups);
  const int P = p.headdim, N = p.d_state;
  const int p0 = static_cast<int>(pb) * kQ, pcols = P - p0 < kQ ? P - p0 : kQ;
  const int64_t nc = p.n_chunks, hp = p.nheads * P, gn = p.ngroups * N;
  float* ws = (back ? p.lam : p.states) + (b * p.nheads + h) * nc * N * P + p0;
  const E* in = static_cast<const E*>(back ? p.C : p.B) + b * p.seqlen * gn + grp * N;
  const E* row = static_cast<const E*>(back ? p.dout : p.x) + b * p.seqlen * hp + h * P + p0;
  const E* zrow = back && p.z ? static_cast<const E*>(p.z) + b * p.seqlen * hp + h * P + p0
                              : nullptr;
  const float* init = p.cut ? nullptr : back ? p.dh_last : p.h0;
  const int col = 16 * pw + l16;  // this lane's channel of the block
  const bool live = col < pcols;
  const int r8 = tid >> 3, c8 = (tid & 7) * 8;
  Oct<IO> io[NB], ro, zo;
  Step st;
  auto fetch = [&](int64_t ch) {
    const int64_t t0 = ch * kQ;
    const bool there = r8 < p.seqlen - t0;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
      io[nb] = load_oct<IO>(in + (t0 + r8) * gn + nb * kQ + c8, there ? N - nb * kQ - c8 : 0);
    ro = load_oct<IO>(row + (t0 + r8) * hp + c8, there ? pcols - c8 : 0);
    if (zrow) zo = load_oct<IO>(zrow + (t0 + r8) * hp + c8, there ? pcols - c8 : 0);
    st = steps<IO>(p, b, h, t0, lane);
  };
  f32x4 S[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int n = 16 * (2 * i + nw) + 4 * g4 + r;
      S[i][r] = init && live && n < N
                    ? init[((b * p.nheads + h) * N + n) * P + p0 + col]
                    : 0.0f;
    }
  auto store = [&](float* out) {
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int n = 16 * (2 * i + nw) + 4 * g4 + r;
        if (live && n < N) out[static_cast<int64_t>(n) * P + col] = S[i][r];
      }
  };
  const int64_t steps_of_walk = p.cut ? 1 : nc;
  const int64_t first = p.cut ? only : back ? nc - 1 : 0;
  fetch(first);
  for (int64_t k = 0; k < steps_of_walk; ++k) {
    const int64_t ch = back ? first - k : first + k;
    if (!p.cut) store(ws + ch * N * P);
    const float decay = st.end;
    __syncthreads();  // the previous chunk's tiles have been read
    // w_s = dt e^{c_end - c_s} forward, e^{c_t} backward
    if (wv == 0) sm.weight[lane] = back ? st.before : st.after * st.dt;
    float v[8];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = io[nb][j];
      put8(sm.in[nb], r8, c8, v);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[j] = ro[j];
      if (zrow) v[j] *= zo[j] * sigmoid_f(zo[j]);
    }
    put8(sm.row, r8, c8, v);
    if (k + 1 < steps_of_walk) fetch(back ? ch - 1 : ch + 1);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NT; ++i) S[i] *= decay;
#pragma unroll 1
    for (int kb = 0; kb < kQ; kb += 16) {
      const Frag x = scaled(down(sm.row, kb, 16 * pw, l16, g4), sm.weight, kb, g4);
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        const int nt = 2 * i + nw;
        S[i] = mac(down(sm.in[nt / 4], kb, 16 * (nt & 3), l16, g4), x, S[i]);
      }
    }
  }
  if (p.cut) {
    store(ws + only * N * P);
    if (tid == 0 && pb == 0)
      p.decay[((back ? p.batch : 0) * p.nheads + b * p.nheads + h) * nc + only] = st.end;
  } else if (back && p.dh0) {
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int n = 16 * (2 * i + nw) + 4 * g4 + r;
        if (live && n < N) p.dh0[((b * p.nheads + h) * N + n) * P + p0 + col] = S[i][r];
      }
  }
}

// ------------------------------------------------------------------ the chunks

constexpr int kThreads = 512;  // eight waves: wave w forms row tile w / 2, column tiles 2 (w % 2)..

struct alignas(16) ChunkSmem {
  float b[kQ * kPitch];     // B of a block of states, (s, n)
  float c[kQ * kPitch];     // C, (t, n)
  float x[kQ * kPitch];     // x of a block of channels, (s, p)
  float gy[kQ * kPitch];    // dout silu(z), (t, p)
  float s[kQ * kPitch];     // S_in, (n, p)
  float lam[kQ * kPitch];   // lam_out, (n, p)
  float m[kQ * kPitch];     // M, (t, s); at the end K
  float dt[kQ], c_hi[kQ], c_lo[kQ];  // step sizes, sums of log2 decays
  float before[kQ], w[kQ];  // e^{c_t}, dt_s e^{c_end - c_s}
  float after[kQ];          // e^{c_end - c_s}
  double erow[2][kQ], ecol[4][kQ];                // sums of E, by the waves' tiles
  float near[2][kQ], far[2][kQ], xv[2][kQ];       // sums over channels: q, p / dt, x . V
  float over[kThreads / 64], diag[4];
};

template <class IO, int NB>
__global__ __launch_bounds__(kThreads) void scan2_chunks_kernel(Scan2BwdArgs p) {
  using E = typename IO::elem;
  __shared__ ChunkSmem sm;
  const int tid = threadIdx.x, wv = tid >> 6, lane = tid & 63, l16 = lane & 15, g4 = lane >> 4;
  const int tr = wv >> 1, tc = 2 * (wv & 1);  // row tile, first column tile
  const int row0 = 16 * tr + 4 * g4;          // first of this lane's four rows of an output tile
  const int P = p.headdim, N = p.d_state;
  const int64_t nc = p.n_chunks, H = p.nheads, hp = H * P, gn = p.ngroups * N;
  int64_t w = blockIdx.x;
  const int64_t split = w % p.splits;
  w /= p.splits;
  const int64_t grp = w % p.ngroups;
  w /= p.ngroups;
  const int64_t ch = w % nc, b = w / nc, t0 = ch * kQ;
  const int rows = p.seqlen - t0 < kQ ? static_cast<int>(p.seqlen - t0) : kQ;
  const int64_t hg = H / p.ngroups;
  const int64_t h_beg = grp * hg + split * hg / p.splits,
                h_end = grp * hg + (split + 1) * hg / p.splits;
  const E* Bg = static_cast<const E*>(p.B) + (b * p.seqlen + t0) * gn + grp * N;
  const E* Cg = static_cast<const E*>(p.C) + (b * p.seqlen + t0) * gn + grp * N;
  const int r8 = tid >> 3, c8 = (tid & 7) * 8;  // this thread's eight values of a tile

  auto stage_bc = [&](int nb) {
    float v[8];
    tile8<IO>(Bg + nb * kQ, gn, rows, N - nb * kQ, r8, c8, v);
    put8(sm.b, r8, c8, v);
    tile8<IO>(Cg + nb * kQ, gn, rows, N - nb * kQ, r8, c8, v);
    put8(sm.c, r8, c8, v);
  };

  // C B^T of the chunk, shared by the heads: this wave's two tiles
  f32x4 G[2] = {}, K[2] = {}, dC[NB][2] = {}, dB[NB][2] = {};
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    if (nb) __syncthreads();
    stage_bc(nb);
    __syncthreads();
#pragma unroll 1
    for (int kb = 0; kb < kQ; kb += 16) {
      const Frag a = along(sm.c, 16 * tr, kb, l16, g4);
#pragma unroll
      for (int i = 0; i < 2; ++i) G[i] = mac(a, along(sm.b, 16 * (tc + i), kb, l16, g4), G[i]);
    }
  }

  for (int64_t h = h_beg; h < h_end; ++h) {
    const int64_t at = (b * p.seqlen + t0) * hp + h * P;
    const float Dh = p.D ? p.D[h] : 0.0f;
    const Step st = steps<IO>(p, b, h, t0, lane);
    __syncthreads();  // the previous head's values have been read
    if (wv == 0) {
      sm.dt[lane] = st.dt;
      sm.c_hi[lane] = st.c_hi;
      sm.c_lo[lane] = st.c_lo;
      sm.before[lane] = st.before;
      sm.after[lane] = st.after;
      sm.w[lane] = st.after * st.dt;
    }
    // x and gy of a block of channels
    auto stage_rows = [&](int p0) {
      float v[8], z[8];
      tile8<IO>(static_cast<const E*>(p.x) + at + p0, hp, rows, P - p0, r8, c8, v);
      put8(sm.x, r8, c8, v);
      tile8<IO>(static_cast<const E*>(p.dout) + at + p0, hp, rows, P - p0, r8, c8, v);
      if (p.z) {
        tile8<IO>(static_cast<const E*>(p.z) + at + p0, hp, rows, P - p0, r8, c8, z);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] *= silu_f(z[j]);
      }
      put8(sm.gy, r8, c8, v);
    };
    // gy X^T
    f32x4 W[2] = {};
    for (int p0 = 0; p0 < P; p0 += kQ) {
      if (p0) __syncthreads();
      stage_rows(p0);
      __syncthreads();
#pragma unroll 1
      for (int kb = 0; kb < kQ; kb += 16) {
        const Frag a = along(sm.gy, 16 * tr, kb, l16, g4);
#pragma unroll
        for (int i = 0; i < 2; ++i) W[i] = mac(a, along(sm.x, 16 * (tc + i), kb, l16, g4), W[i]);
      }
    }
    // M to LDS, K into its sum, the sums of E and the diagonal of gy X^T
    double er[4] = {}, ec[2] = {};
    float diag = 0.0f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int s = 16 * (tc + i) + l16;
      const float ch = sm.c_hi[s], cl = sm.c_lo[s], dts = sm.dt[s];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int t = row0 + r;
        const float seg = s <= t ? exp2_diff(sm.c_hi[t], sm.c_lo[t], ch, cl) : 0.0f;
        const float m = s <= t ? G[i][r] * seg : 0.0f;
        const float k = s <= t ? W[i][r] * seg * dts : 0.0f;
        const float e = s < t ? W[i][r] * dts * m : 0.0f;
        sm.m[t * kPitch + s] = m;
        K[i][r] += k;
        er[r] += e;
        ec[i] += e;
        if (s == t) diag += W[i][r];
      }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      er[r] = sum16(er[r]);
      if (l16 == 0) sm.erow[wv & 1][row0 + r] = er[r];
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      ec[i] = sum_rows(ec[i]);
      if (g4 == 0) sm.ecol[tr][16 * (tc + i) + l16] = ec[i];
    }
    diag = sum64(diag);
    // (the diagonal of row tile tr lies in the wave that holds column tile tr)
    if (lane == 0 && (tr >> 1) == (wv & 1)) sm.diag[tr] = diag;

    float near[4] = {}, far[4] = {}, xv[4] = {}, over = 0.0f;
    for (int p0 = 0; p0 < P; p0 += kQ) {
      const int pcols = P - p0 < kQ ? P - p0 : kQ;
      f32x4 Y[2] = {}, V[2] = {};  // C S_in and B lam_out
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        __syncthreads();
        if (P > kQ && nb == 0) stage_rows(p0);
        if (NB > 1) stage_bc(nb);
        {
          const int n = nb * kQ + r8;
          const int64_t off = (((b * H + h) * nc + ch) * N + nb * kQ) * P + p0;
          float v[8], q[8];
          const int have = n < N ? pcols - c8 : 0;
          load8<F32>(p.states + off + static_cast<int64_t>(r8) * P + c8, have, v);
          load8<F32>(p.lam + off + static_cast<int64_t>(r8) * P + c8, have, q);
          put8(sm.s, r8, c8, v);
          put8(sm.lam, r8, c8, q);
#pragma unroll
          for (int j = 0; j < 8; ++j) over = fmaf(v[j], q[j], over);
        }
        __syncthreads();
        const float bt = sm.before[16 * tr + l16], wt = sm.w[16 * tr + l16];
#pragma unroll 1
        for (int kb = 0; kb < kQ; kb += 16) {
          const Frag cf = along(sm.c, 16 * tr, kb, l16, g4), bf = along(sm.b, 16 * tr, kb, l16, g4);
          const Frag gf = along(sm.gy, 16 * tr, kb, l16, g4) * bt;
          const Frag xf = along(sm.x, 16 * tr, kb, l16, g4) * wt;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            Y[i] = mac(cf, down(sm.s, kb, 16 * (tc + i), l16, g4), Y[i]);
            V[i] = mac(bf, down(sm.lam, kb, 16 * (tc + i), l16, g4), V[i]);
            dC[nb][i] = mac(gf, along(sm.s, 16 * (tc + i), kb, l16, g4), dC[nb][i]);
            dB[nb][i] = mac(xf, along(sm.lam, 16 * (tc + i), kb, l16, g4), dB[nb][i]);
          }
        }
      }
      // the carried parts are scaled by their rows, and their share of dl and ddt summed
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int t = row0 + r, c = 16 * (tc + i) + l16;
          Y[i][r] *= sm.before[t];
          V[i][r] *= sm.after[t];
          near[r] = fmaf(sm.gy[t * kPitch + c], Y[i][r], near[r]);
          far[r] = fmaf(sm.x[t * kPitch + c], V[i][r], far[r]);
        }
      // the chunk's own part: M (dt X) over s <= t, M^T gy over t >= s
#pragma unroll 1
      for (int kb = 0; kb < kQ; kb += 16) {
        if (kb <= 16 * tr) {
          const Frag a = scaled(along(sm.m, 16 * tr, kb, l16, g4), sm.dt, kb, g4);
#pragma unroll
          for (int i = 0; i < 2; ++i)
            Y[i] = mac(a, down(sm.x, kb, 16 * (tc + i), l16, g4), Y[i]);
        }
        if (kb >= 16 * tr) {
          const Frag a = down(sm.m, kb, 16 * tr, l16, g4);
#pragma unroll
          for (int i = 0; i < 2; ++i)
            V[i] = mac(a, down(sm.gy, kb, 16 * (tc + i), l16, g4), V[i]);
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int t = row0 + r, c = 16 * (tc + i) + l16;
          const float x = sm.x[t * kPitch + c];
          xv[r] = fmaf(x, V[i][r], xv[r]);
          if (t < rows && c < pcols) {
            const int64_t o = at + t * hp + p0 + c;
            static_cast<E*>(p.dx)[o] =
                IO::from_float(fmaf(sm.dt[t], V[i][r], Dh * sm.gy[t * kPitch + c]));
            if (p.z) {
              const float z = IO::widen(static_cast<const E*>(p.z)[o]);
              const float go = IO::widen(static_cast<const E*>(p.dout)[o]);
              const float sg = sigmoid_f(z);
              static_cast<E*>(p.dz)[o] = IO::from_float(
                  go * fmaf(Dh, x, Y[i][r]) * (sg * fmaf(z, 1.0f - sg, 1.0f)));
            }
          }
        }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      near[r] = sum16(near[r]);
      far[r] = sum16(far[r]);
      xv[r] = sum16(xv[r]);
      if (l16 == 0) {
        sm.near[wv & 1][row0 + r] = near[r];
        sm.far[wv & 1][row0 + r] = far[r];
        sm.xv[wv & 1][row0 + r] = xv[r];
      }
    }
    over = sum64(over);
    if (lane == 0) sm.over[wv] = over;
    __syncthreads();
    if (wv == 0) {
      const float q = sm.near[0][lane] + sm.near[1][lane];
      const double ps = static_cast<double>(st.dt) * (sm.far[0][lane] + sm.far[1][lane]);
      const double in = (sm.ecol[0][lane] + sm.ecol[1][lane]) +
                        (sm.ecol[2][lane] + sm.ecol[3][lane]);
      const double out = sm.erow[0][lane] + sm.erow[1][lane];
      // inclusive sums in float64; what lies before a step is the sum less its own
      const double flow = in - out + ps, before = scan64(flow) - flow;
      const double upto = scan64(q), since = last_lane(upto) - (upto - q);
      float ov = 0.0f;
      for (int k = 0; k < kThreads / 64; ++k) ov += sm.over[k];
      const float dl = static_cast<float>(before + since + static_cast<double>(st.end) * ov);
      float ddt = fmaf(p.A[h], dl, sm.xv[0][lane] + sm.xv[1][lane]);
      ddt *= st.slope;
      if (lane >= rows) ddt = 0.0f;
      else
        static_cast<E*>(p.ddt)[(b * p.seqlen + t0 + lane) * H + h] = IO::from_float(ddt);
      const float sa = sum64(st.dt * dl), sb = sum64(ddt);
      if (lane == 0) {
        float* line = p.head_part + (b * nc + ch) * 3 * H + h;
        line[0] = sa;
        line[H] = (sm.diag[0] + sm.diag[1]) + (sm.diag[2] + sm.diag[3]);
        line[2 * H] = sb;
      }
    }
  }

  // dC = K B + ..., dB = K^T C + ...
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int r = 0; r < 4; ++r) sm.m[(row0 + r) * kPitch + 16 * (tc + i) + l16] = K[i][r];
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    if (nb) __syncthreads();
    stage_bc(nb);
    __syncthreads();
#pragma unroll 1
    for (int kb = 0; kb < kQ; kb += 16) {
      if (kb <= 16 * tr) {
        const Frag a = along(sm.m, 16 * tr, kb, l16, g4);
#pragma unroll
        for (int i = 0; i < 2; ++i)
          dC[nb][i] = mac(a, down(sm.b, kb, 16 * (tc + i), l16, g4), dC[nb][i]);
      }
      if (kb >= 16 * tr) {
        const Frag a = down(sm.m, kb, 16 * tr, l16, g4);
#pragma unroll
        for (int i = 0; i < 2; ++i)
          dB[nb][i] = mac(a, down(sm.c, kb, 16 * (tc + i), l16, g4), dB[nb][i]);
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int t = row0 + r, n = nb * kQ + 16 * (tc + i) + l16;
        if (t < rows && n < N) {
          const int64_t o = ((b * p.seqlen + t0 + t) * p.ngroups + grp) * N + n;
          if (p.splits == 1) {
            static_cast<E*>(p.dB)[o] = IO::from_float(dB[nb][i][r]);
            static_cast<E*>(p.dC)[o] = IO::from_float(dC[nb][i][r]);
          } else {
            const int64_t all = p.batch * p.seqlen * gn;
            p.bc_part[split * 2 * all + o] = dB[nb][i][r];
            p.bc_part[split * 2 * all + all + o] = dC[nb][i][r];
          }
        }
      }
  }
}

// Where walks are cut, S' = decay S + part along the chunks: one value of a state per lane and
// direction, whose slots hold the chunks' own parts and take what lies before (behind) each chunk.
// Latency bounds it, so eight chunks' parts are in flight (5 us for 13 chunks of 18 heads of 48 x 40).
template <bool TILED>
__global__ __launch_bounds__(256) void scan2_join_kernel(Scan2BwdArgs p) {
  const int64_t np = static_cast<int64_t>(p.d_state) * p.headdim, heads = p.batch * p.nheads;
  const int64_t all = heads * np, nc = p.n_chunks;
  int64_t i = blockIdx.x * 256ll + threadIdx.x;
  if (i >= 2 * all) return;
  const bool back = i >= all;
  if (back) i -= all;
  const int64_t bh = i / np;
  const int e = static_cast<int>(i - bh * np);
  // the value's place in h0, dh_last and dh0: (state, channel)
  const int64_t at = TILED ? bh * np + (e / (16 * p.headdim) * 16 + e % 16) * p.headdim +
                                 e / 16 % p.headdim
                           : i;
  const float* init = back ? p.dh_last : p.h0;
  float* slot = (back ? p.lam : p.states) + bh * nc * np + e;
  const float* decay = p.decay + ((back ? heads : 0) + bh) * nc;
  float S = init ? init[at] : 0.0f;
  constexpr int kAhead = 8;
  for (int64_t k = 0; k < nc; k += kAhead) {
    float part[kAhead], d[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      if (k + j < nc) {
        const int64_t ch = back ? nc - 1 - (k + j) : k + j;
        part[j] = slot[ch * np];
        d[j] = decay[ch];
      }
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      if (k + j < nc) {
        const int64_t ch = back ? nc - 1 - (k + j) : k + j;
        slot[ch * np] = S;
        S = fmaf(d[j], S, part[j]);
      }
  }
  if (back && p.dh0) p.dh0[at] = S;
}

// dB and dC: the runs of heads added in order.
template <class IO>
__global__ __launch_bounds__(256) void scan2_runs_kernel(const float* part, int64_t n,
                                                         int64_t splits,
                                                         typename IO::elem* dB,
                                                         typename IO::elem* dC) {
  for (int64_t i = (blockIdx.x * 256ll + threadIdx.x) * 8; i < 2 * n; i += gridDim.x * 2048ll) {
    float s[8];
    const int64_t left = 2 * n - i;
    const int have = left < 8 ? static_cast<int>(left) : 8;
    load8<F32>(part + i, have, s);
    for (int64_t k = 1; k < splits; ++k) {
      float v[8];
      load8<F32>(part + k * 2 * n + i, have, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) s[j] += v[j];
    }
    if (i + 8 <= n) store8<IO>(dB + i, 8, s);
    else if (i >= n) store8<IO>(dC + (i - n), have, s);
    else
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (i + j < n) dB[i + j] = IO::from_float(s[j]);
        else if (j < have) dC[i + j - n] = IO::from_float(s[j]);
      }
  }
}

template <class IO, int NB>
hipError_t launch_nb(const Scan2BwdArgs& a, hipStream_t stream) {
  const dim3 walks(
      static_cast<unsigned>(2 * a.batch * a.nheads * a.n_pblk * (a.cut ? a.n_chunks : 1)));
  hipLaunchKernelGGL((scan2_states_kernel<IO, NB>), walks, dim3(512), 0, stream, a);
  if (a.cut) {
    const hipError_t e = launch_scan2_join(a, false, stream);
    if (e != hipSuccess) return e;
  }
  const dim3 chunks(static_cast<unsigned>(a.batch * a.n_chunks * a.ngroups * a.splits));
  hipLaunchKernelGGL((scan2_chunks_kernel<IO, NB>), chunks, dim3(kThreads), 0, stream, a);
  return hipGetLastError();
}

template <class IO>
hipError_t launch_io(const Scan2BwdArgs& a, hipStream_t stream) {
  using E = typename IO::elem;
  hipError_t e;
  if (scan2_bwd_mfma_supported(a, sizeof(E) == 2)) e = launch_scan2_bwd_mfma(a, stream);
  else switch ((a.d_state + kQ - 1) / kQ) {
    case 1: e = launch_nb<IO, 1>(a, stream); break;
    case 2: e = launch_nb<IO, 2>(a, stream); break;
    case 3: e = launch_nb<IO, 3>(a, stream); break;
    default: e = launch_nb<IO, 4>(a, stream); break;
  }
  if (e != hipSuccess) return e;
  if (a.splits > 1) {
    const int64_t n = a.batch * a.seqlen * a.ngroups * a.d_state;
    const int64_t blocks = (2 * n + 2047) / 2048;
    hipLaunchKernelGGL(scan2_runs_kernel<IO>, dim3(static_cast<unsigned>(blocks < 4096 ? blocks : 4096)),
                       dim3(256), 0, stream, a.bc_part, n, a.splits, static_cast<E*>(a.dB),
                       static_cast<E*>(a.dC));
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  ColumnSums c{};
  c.lines = a.batch * a.n_chunks;
  c.stride = 3 * a.nheads;
  c.cols = a.nheads;
  c.add(a.head_part, a.dA, 1);
  c.add(a.head_part + a.nheads, a.dD, 1);
  c.add(a.head_part + 2 * a.nheads, a.ddt_bias, 1);
  return launch_column_sums(c, stream);
}

int64_t round16(int64_t floats) { return (floats + 3) / 4 * 4; }

}  // namespace

hipError_t launch_scan2_join(const Scan2BwdArgs& a, bool tiled, hipStream_t stream) {
  const int64_t n = 2 * a.batch * a.nheads * a.d_state * a.headdim;
  const dim3 grid(static_cast<unsigned>((n + 255) / 256));
  if (tiled) hipLaunchKernelGGL(scan2_join_kernel<true>, grid, dim3(256), 0, stream, a);
  else hipLaunchKernelGGL(scan2_join_kernel<false>, grid, dim3(256), 0, stream, a);
  return hipGetLastError();
}

// Walks too few to fill the 256 CUs are cut into their chunks, which costs one more launch and the
// states read and written once more.  The whole call, walks whole -> cut: bf16, headdim 64, d_state
// 128, one batch row: 8 heads x 4096 steps 196 -> 74 us, 24 x 4096 239 -> 153, 48 x 2048 165 -> 149,
// 48 x 512 73 -> 70, 64 x 4096 380 -> 394, 24 x 256 48 -> 49, 24 x 128 41 -> 44; float32: 3 x 777,
// 6 heads of 48 x 40, 73 -> 49, 1 x 16384, 24 heads of 64 x 128, 1820 -> 1150, 1 x 4096, 64 heads,
// 765 -> 785.
// Walks of more chunks than a launch has workgroups for stay whole.
constexpr int64_t kCutWalks = 96, kCutChunks = 4;
bool scan2_bwd_cut(int64_t heads, int64_t n_pblk, int64_t nc) {
  const int64_t walks = 2 * heads * n_pblk;
  return walks <= kCutWalks && nc >= kCutChunks && walks * nc <= kScan2BwdMaxWalks;
}

// Runs of heads: a workgroup for each of the 256 CUs (one fits a CU), at most a head each.  The rule
// counts workgroups, not their rounds over the CUs, so that a little more than a multiple of 256 units
// costs a whole round more.  Backward of 80 heads of 64 x 128 bf16, one group, us for a thousand steps:
// 4 x 4096 (256 units) 83, 8 x 4096 79, 6 x 4096 97, 5 x 4096 111, 4 x 4160 130; 3 x 4096 (192 units) 97,
// 2 x 4160 138, 1 x 4160 153.
int64_t scan2_bwd_splits(int64_t batch, int64_t seqlen, int64_t nheads, int64_t ngroups) {
  const int64_t units = batch * ((seqlen + kQ - 1) / kQ) * ngroups, hg = nheads / ngroups;
  const int64_t want = (256 + units - 1) / units;
  return want < hg ? want : hg;
}

int64_t scan2_bwd_ws_floats(int64_t batch, int64_t seqlen, int64_t nheads, int64_t headdim,
                            int64_t ngroups, int64_t d_state, Scan2BwdArgs* a, float* ws) {
  const int64_t nc = (seqlen + kQ - 1) / kQ;
  const int64_t splits = scan2_bwd_splits(batch, seqlen, nheads, ngroups);
  const int64_t states = round16(batch * nheads * nc * d_state * headdim);
  const int64_t heads = round16(batch * nc * 3 * nheads);
  const int64_t runs = splits > 1 ? round16(splits * 2 * batch * seqlen * ngroups * d_state) : 0;
  const int64_t n_pblk = (headdim + kQ - 1) / kQ;
  const bool cut = scan2_bwd_cut(batch * nheads, n_pblk, nc);
  const int64_t decays = cut ? 2 * batch * nheads * nc : 0;
  if (a) {
    a->n_chunks = nc;
    a->splits = splits;
    a->n_pblk = n_pblk;
    a->cut = cut;
    a->states = ws;
    a->lam = ws + states;
    a->head_part = a->lam + states;
    a->bc_part = a->head_part + heads;
    a->decay = a->bc_part + runs;
  }
  return 2 * states + heads + runs + decays;
}

hipError_t launch_scan2_bwd(const Scan2BwdArgs& a, bool bf16, hipStream_t stream) {
  return bf16 ? launch_io<BF16>(a, stream) : launch_io<F32>(a, stream);
}

}  // namespace ss
