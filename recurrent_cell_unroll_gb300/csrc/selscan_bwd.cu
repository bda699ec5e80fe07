// Selective scan, backward (selscan.cuh has the mathematics and the layout).
//
//   gy = dy silu(z), s_t = sum_n c h_t + d x,     dz = dy s silu'(z)
//   e_t[n] = gy_t c_t[n] + a_{t+1}[n] e_{t+1}[n]  (the gradient reaching a state)
//   dx = delta sum_n e b + gy d,   ddelta = sum_n e (a A h_{t-1} + b x)
//   db_t[n] = sum_ch e delta x,    dc_t[n] = sum_ch gy h_t,   da_log = A sum e a h_{t-1} delta
//
// A block takes the chunks of 32 steps from the last to the first.  In a chunk it
// runs the states forward from the kept ones, leaving those before every fourth
// step in shared memory, then takes four steps at a time backwards: their states
// and decays once more, in registers, and the gradients against them.
//
// The sums over channels (db, dc) are what costs beside that: a thread has two
// channels, whose products it adds first, and the warp's lanes exchange theirs
// through the checkpoint of the four steps, which has been read by then.
#include "selscan.cuh"

namespace rcu {
namespace {

using namespace selscan;

constexpr int TILE = CHUNK;                // steps of a tile: those between two kept states
constexpr int SUB = 4, SUBS = TILE / SUB;  // steps in registers, and groups of them in a chunk
constexpr int S = 8, K = 2;                // states and channels of a thread
constexpr int SLOT = 32 * K * S;           // floats of a warp's checkpoint

struct Args {
  ScanBwd p;
  int groups, warps;     // blocks of channels; warps of a block
  Segments seg;
  const float *enter;    // [seg][B][H][N]: gradients that enter each segment, or dh_n
  float *part_bc;        // [groups][T][B][2][N], or NULL
  float *part;           // [B * seg][H N | H | H], or NULL
  bool wide_states;
};

template <int LANES>
constexpr int slots() { return LANES == 8 ? SUBS : SUBS - 1; }
template <int LANES>
constexpr int channels() { return 32 / LANES * K; }  // of a warp
template <int LANES>
size_t shared_bytes(int warps) {
  const size_t cc = (size_t)channels<LANES>() * warps;
  return (size_t)warps * slots<LANES>() * SLOT * 4 + 3 * TILE * cc * 4 + 2 * TILE * LANES * S * 4;
}

template <typename T, int LANES>
__global__ void __launch_bounds__(128, 2) scan_bwd_kernel(const Args a, int *err) {
  constexpr int NP = S * LANES, WC = channels<LANES>(), SLOTS = slots<LANES>();
  const ScanBwd &p = a.p;
  const ScanIn &in = p.in;
  const int NT = a.warps * 32, CC = WC * a.warps;
  extern __shared__ float4 shared4[];
  float *check = reinterpret_cast<float *>(shared4);    // [warps][SLOTS][SLOT]
  float *s_delta = check + a.warps * SLOTS * SLOT;      // [TILE][CC]
  float *s_u = s_delta + TILE * CC;                     // delta x
  float *s_gy = s_u + TILE * CC;
  float *s_b = s_gy + TILE * CC;                        // [TILE][NP]
  float *s_c = s_b + TILE * NP;

  const int group = blockIdx.x % a.groups;
  const int b = (int)(blockIdx.x / a.groups % in.B), seg = (int)(blockIdx.x / a.groups / in.B);
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32, l = lane % LANES, cl = lane / LANES;
  const int ch0 = group * CC, own = warp * WC + cl * K;  // the thread's channels in the block
  const int n0 = l * S;
  const int64_t table = (int64_t)in.B * in.H * in.N;
  const int n = row_length(in.lengths, b, in.T, err);
  const int t0 = seg * a.seg.len, t1 = min(t0 + a.seg.len, in.T), end = min(t1, n);
  float *mine = check + warp * SLOTS * SLOT;

  int here[K];  // states that exist
  int64_t at[K];
  F2 A2[K][S / 2], e[K][S / 2], dA[K][S / 2];
#pragma unroll
  for (int c = 0; c < K; ++c) {
    const int ch = ch0 + own + c;
    here[c] = ch < in.H ? min(max(in.N - n0, 0), S) : 0;
    at[c] = ((int64_t)b * in.H + ch) * in.N + n0;
    float v[S];
    load_states(in.a_log + (int64_t)ch * in.N + n0, here[c], a.wide_states, v);
#pragma unroll
    for (int k = 0; k < S; ++k) v[k] = k < here[c] ? rate2(v[k]) : 0.f;
#pragma unroll
    for (int k = 0; k < S / 2; ++k) A2[c][k] = f2(v[2 * k], v[2 * k + 1]);
#pragma unroll
    for (int k = 0; k < S; ++k) v[k] = 0.f;
    if (a.enter) load_states(a.enter + (a.seg.n > 1 ? seg * table : 0) + at[c], here[c], a.wide_states, v);
#pragma unroll
    for (int k = 0; k < S / 2; ++k) {
      e[c][k] = f2(v[2 * k], v[2 * k + 1]);
      dA[c][k] = f2(0.f);
    }
  }
  // the channel whose sums over states this lane ends up with, if it is one of the
  // first two lanes of its channels (with one lane: both)
  constexpr int OWN = LANES == 1 ? K : 1;
  float dd[OWN] = {}, ddtb[OWN] = {};

  const T *x = static_cast<const T *>(in.x.p) + b * in.x.sb + ch0;
  const T *dt = static_cast<const T *>(in.dt.p) + b * in.dt.sb + ch0;
  const T *z = in.z.p ? static_cast<const T *>(in.z.p) + b * in.z.sb + ch0 : nullptr;
  const T *dy = static_cast<const T *>(p.dy.p) + b * p.dy.sb + ch0;
  const T *bw = static_cast<const T *>(in.b.p) + b * in.b.sb;
  const T *cw = static_cast<const T *>(in.c.p) + b * in.c.sb;
  T *dx = p.dx.p ? static_cast<T *>(p.dx.p) + b * p.dx.sb + ch0 : nullptr;
  T *ddt = p.ddt.p ? static_cast<T *>(p.ddt.p) + b * p.ddt.sb + ch0 : nullptr;
  T *dz = p.dz.p && z ? static_cast<T *>(p.dz.p) + b * p.dz.sb + ch0 : nullptr;

  auto load_pairs_of = [&](const float *row, F2 (&v)[S / 2]) { load_pairs<S / 2>(row + n0, v); };
  // h after a step, from the state before it; the decay where it is wanted
  auto step = [&](int t, const F2 (&w)[S / 2], F2 (&h)[K][S / 2], F2 (*decay)[S / 2]) {
    const float2 d = *reinterpret_cast<const float2 *>(s_delta + t * CC + own);
    const float2 u = *reinterpret_cast<const float2 *>(s_u + t * CC + own);
#pragma unroll
    for (int c = 0; c < K; ++c) {
      const F2 d2 = f2(c ? d.y : d.x), u2 = f2(c ? u.y : u.x);
#pragma unroll
      for (int q = 0; q < S / 2; ++q) {
        const F2 r = ex2_2(mul2(d2, A2[c][q]));
        if (decay) decay[c][q] = r;
        h[c][q] = fma2(r, h[c][q], mul2(u2, w[q]));
      }
    }
  };
  auto save = [&](int slot, const F2 (&h)[K][S / 2]) {
    ulonglong2 *to = reinterpret_cast<ulonglong2 *>(mine + slot * SLOT) + lane;
#pragma unroll
    for (int q = 0; q < K * S / 4; ++q)
      to[q * 32] = make_ulonglong2(h[q / 2][q % 2 * 2], h[q / 2][q % 2 * 2 + 1]);
  };
  auto restore = [&](int slot, F2 (&h)[K][S / 2]) {
    const ulonglong2 *from = reinterpret_cast<const ulonglong2 *>(mine + slot * SLOT) + lane;
#pragma unroll
    for (int q = 0; q < K * S / 4; ++q) {
      const ulonglong2 v = from[q * 32];
      h[q / 2][q % 2 * 2] = v.x;
      h[q / 2][q % 2 * 2 + 1] = v.y;
    }
  };
  auto first_states = [&](int base, F2 (&h)[K][S / 2]) {
#pragma unroll
    for (int c = 0; c < K; ++c) {
      float v[S];
      load_states(p.states + (base / TILE) * table + at[c], here[c], a.wide_states, v);
#pragma unroll
      for (int k = 0; k < S / 2; ++k) h[c][k] = f2(v[2 * k], v[2 * k + 1]);
    }
  };

  const int tiles = t0 < end ? ceil_div(end - t0, TILE) : 0;
  for (int k = tiles - 1; k >= 0; --k) {
    const int base = t0 + k * TILE;
    for (int i = tid; i < TILE * CC; i += NT) {
      const int t = i / CC, c = i % CC;
      float delta = 0.f, u = 0.f, gy = 0.f;
      if (base + t < end && ch0 + c < in.H) {
        const int64_t s = base + t;
        delta = softplus(to_f(dt[s * in.dt.st + c]) + (in.dt_bias ? in.dt_bias[ch0 + c] : 0.f));
        u = delta * to_f(x[s * in.x.st + c]);
        gy = to_f(dy[s * p.dy.st + c]);
        if (z) {
          const float v = to_f(z[s * in.z.st + c]);
          gy *= v * sigmoid(v);
        }
      }
      s_delta[i] = delta;
      s_u[i] = u;
      s_gy[i] = gy;
    }
    for (int i = tid; i < TILE * NP; i += NT) {
      const int t = i / NP, m = i % NP;
      const bool there = base + t < end && m < in.N;
      s_b[i] = there ? to_f(bw[(base + t) * in.b.st + m]) : 0.f;
      s_c[i] = there ? to_f(cw[(base + t) * in.c.st + m]) : 0.f;
    }
    F2 h[K][S / 2];
    first_states(base, h);
    __syncthreads();
    const int steps = min(TILE, end - base), subs = ceil_div(steps, SUB);
    if (SLOTS == SUBS) save(0, h);
    for (int t = 0; t < (subs - 1) * SUB; ++t) {
      F2 w[S / 2];
      load_pairs_of(s_b + t * NP, w);
      step(t, w, h, nullptr);
      if (t % SUB == SUB - 1) save(t / SUB + SLOTS - (SUBS - 1), h);
    }
    for (int sub = subs - 1; sub >= 0; --sub) {
      const int slot = sub + SLOTS - SUBS;  // where its checkpoint is; before the first: none
      F2 before[SUB][K][S / 2], decay[SUB][K][S / 2];
      if (slot >= 0) {
        if (sub < subs - 1) restore(slot, h);  // the last one's is at hand
      } else if (subs > 1) {
        first_states(base, h);
      }
#pragma unroll
      for (int j = 0; j < SUB; ++j) {
#pragma unroll
        for (int c = 0; c < K; ++c)
#pragma unroll
          for (int q = 0; q < S / 2; ++q) before[j][c][q] = h[c][q];
        F2 w[S / 2];
        load_pairs_of(s_b + (sub * SUB + j) * NP, w);
        step(sub * SUB + j, w, h, decay[j]);
      }
      // the lanes' exchange is where the checkpoint was, or, of the first steps, the
      // next one's, whose db and dc have been added by then
      float *room = mine + max(slot, 0) * SLOT;
      (void)room;
      __syncwarp();
#pragma unroll
      for (int j = SUB - 1; j >= 0; --j) {
        const int t = sub * SUB + j;
        F2 w[S / 2], v[S / 2], db[S / 2], dc[S / 2];
        load_pairs_of(s_b + t * NP, w);
        load_pairs_of(s_c + t * NP, v);
        const float2 d = *reinterpret_cast<const float2 *>(s_delta + t * CC + own);
        const float2 u = *reinterpret_cast<const float2 *>(s_u + t * CC + own);
        const float2 g = *reinterpret_cast<const float2 *>(s_gy + t * CC + own);
        float out[K], du[K], dlog[K];
#pragma unroll
        for (int c = 0; c < K; ++c) {
          const F2 d2 = f2(c ? d.y : d.x), u2 = f2(c ? u.y : u.x), g2 = f2(c ? g.y : g.x);
          F2 so, sd, sl;
#pragma unroll
          for (int q = 0; q < S / 2; ++q) {
            e[c][q] = fma2(g2, v[q], e[c][q]);
            so = q ? fma2(h[c][q], v[q], so) : mul2(h[c][q], v[q]);
            sd = q ? fma2(e[c][q], w[q], sd) : mul2(e[c][q], w[q]);
            db[q] = c ? fma2(e[c][q], u2, db[q]) : mul2(e[c][q], u2);
            dc[q] = c ? fma2(h[c][q], g2, dc[q]) : mul2(h[c][q], g2);
            e[c][q] = mul2(e[c][q], decay[j][c][q]);
            const F2 r = mul2(e[c][q], before[j][c][q]);
            sl = q ? fma2(r, A2[c][q], sl) : mul2(r, A2[c][q]);
            dA[c][q] = fma2(r, d2, dA[c][q]);
            h[c][q] = before[j][c][q];
          }
          out[c] = lo(so) + hi(so);
          du[c] = lo(sd) + hi(sd);
          dlog[c] = lo(sl) + hi(sl);
        }
        // sums over the states: lane 0 of a channel pair gets the first one's, lane 1
        // the second's
        if (LANES > 1) {
          float *const sums[3] = {out, du, dlog};
#pragma unroll
          for (int q = 0; q < 3; ++q) {
            const float keep = l & 1 ? sums[q][1] : sums[q][0], give = l & 1 ? sums[q][0] : sums[q][1];
            float s = keep + __shfl_xor_sync(0xffffffffu, give, 1);
#pragma unroll
            for (int o = 2; o < LANES; o *= 2) s += __shfl_xor_sync(0xffffffffu, s, o);
            sums[q][0] = s;
          }
        }
        if (l < K && t < steps) {
#pragma unroll
          for (int c = 0; c < OWN; ++c) {
            const int ch = own + (LANES == 1 ? c : l);
            if (ch0 + ch < in.H) {
              const int64_t s = base + t;
              const float xv = to_f(x[s * in.x.st + ch]);
              const float delta = s_delta[t * CC + ch], gy = s_gy[t * CC + ch];
              const float skip = p.in.d ? in.d[ch0 + ch] : 0.f;
              if (dx) dx[s * p.dx.st + ch] = from_f<T>(fmaf(du[c], delta, gy * skip));
              const float logit = to_f(dt[s * in.dt.st + ch]) + (in.dt_bias ? in.dt_bias[ch0 + ch] : 0.f);
              // A2 is in units of log2(e)
              const float gdt = fmaf(dlog[c], 1.f / LOG2E, du[c] * xv) * sigmoid(logit);
              if (ddt) ddt[s * p.ddt.st + ch] = from_f<T>(gdt);
              if (dz) {
                const float zv = to_f(z[s * in.z.st + ch]), sg = sigmoid(zv);
                const float total = p.in.d ? fmaf(skip, xv, out[c]) : out[c];
                dz[s * p.dz.st + ch] =
                    from_f<T>(to_f(dy[s * p.dy.st + ch]) * total * sg * fmaf(zv, 1.f - sg, 1.f));
              }
              ddtb[c] += gdt;
              dd[c] = fmaf(gy, xv, dd[c]);
            }
          }
        }
        if (a.part_bc) {
          // sums over the warp's channels, then over the warps below
          float val[2 * S];
#pragma unroll
          for (int q = 0; q < S / 2; ++q) {
            val[2 * q] = lo(db[q]), val[2 * q + 1] = hi(db[q]);
            val[S + 2 * q] = lo(dc[q]), val[S + 2 * q + 1] = hi(dc[q]);
          }
#pragma unroll
          for (int q = 0; q < 2 * S; ++q)
#pragma unroll
            for (int o = LANES; o < 32; o *= 2) val[q] += __shfl_xor_sync(0xffffffffu, val[q], o);
          // a group of four steps needs 4 * 2 * NP floats of its slot
          float *to = mine + max(slot, 0) * SLOT + (slot < 0 ? SUB * 2 * NP : 0) + j * 2 * NP;
          if (cl == 0) {
#pragma unroll
            for (int q = 0; q < S; ++q) {
              to[n0 + q] = val[q];
              to[NP + n0 + q] = val[S + q];
            }
          }
        }
      }
    }
    __syncthreads();
    if (a.part_bc) {
      float *to = a.part_bc + (int64_t)group * in.T * in.B * 2 * in.N;
      for (int i = tid; i < steps * 2 * NP; i += NT) {
        const int t = i / (2 * NP), m = i % (2 * NP), sub = t / SUB, slot = sub + SLOTS - SUBS;
        const float *from = check + max(slot, 0) * SLOT + (slot < 0 ? SUB * 2 * NP : 0) + t % SUB * 2 * NP + m;
        float s = 0.f;
        for (int w = 0; w < a.warps; ++w) s += from[w * SLOTS * SLOT];
        if (m % NP < in.N)
          to[((int64_t)(base + t) * in.B + b) * 2 * in.N + (m / NP) * in.N + m % NP] = s;
      }
      __syncthreads();
    }
  }
  // past the row's end
  for (int64_t i = tid; i < (int64_t)(t1 - max(t0, end)) * CC; i += NT) {
    const int64_t t = max(t0, end) + i / CC;
    const int c = (int)(i % CC);
    if (ch0 + c >= in.H) continue;
    if (dx) dx[t * p.dx.st + c] = from_f<T>(0.f);
    if (ddt) ddt[t * p.ddt.st + c] = from_f<T>(0.f);
    if (dz) dz[t * p.dz.st + c] = from_f<T>(0.f);
  }
  auto put = [&](float *to, const F2 (&v)[S / 2], int k, float scale2, const F2 *scale) {
    float out[S];
#pragma unroll
    for (int q = 0; q < S / 2; ++q) {
      out[2 * q] = lo(v[q]) * (scale ? lo(scale[q]) * scale2 : 1.f);
      out[2 * q + 1] = hi(v[q]) * (scale ? hi(scale[q]) * scale2 : 1.f);
    }
    store_states(to, k, false, out);
  };
#pragma unroll
  for (int c = 0; c < K; ++c) {
    if (seg == 0 && p.dh0) put(p.dh0 + at[c], e[c], here[c], 1.f, nullptr);
    if (a.part) {
      float *to = a.part + ((int64_t)seg * in.B + b) * in.H * (in.N + 2);
      put(to + (int64_t)(ch0 + own + c) * in.N + n0, dA[c], here[c], 1.f / LOG2E, A2[c]);
    }
  }
  if (a.part && l < K) {
#pragma unroll
    for (int c = 0; c < OWN; ++c) {
      const int ch = ch0 + own + (LANES == 1 ? c : l);
      if (ch < in.H) {
        float *to = a.part + ((int64_t)seg * in.B + b) * in.H * (in.N + 2) + (int64_t)in.H * in.N;
        to[ch] = dd[c];
        to[in.H + ch] = ddtb[c];
      }
    }
  }
}

int lanes_of(int N) { return N <= 8 ? 1 : N <= 16 ? 2 : N <= 32 ? 4 : 8; }
template <typename F>
cudaError_t by_lanes(int N, F f) {
  switch (lanes_of(N)) {
    case 1: return f(std::integral_constant<int, 1>());
    case 2: return f(std::integral_constant<int, 2>());
    case 4: return f(std::integral_constant<int, 4>());
    default: return f(std::integral_constant<int, 8>());
  }
}

// db and dc from the blocks' sums, [groups][T][B][2][N]: a thread a value.
template <typename T>
__global__ void __launch_bounds__(256) sum_bc_kernel(const float *part, int groups, int T_, int B, int N,
                                                     const int32_t *lengths, SeqOut db, SeqOut dc) {
  wait_for_previous();
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, all = (int64_t)T_ * B * 2 * N;
  if (i >= all) return;
  const int m = (int)(i % (2 * N)), b = (int)(i / (2 * N) % B);
  const int64_t t = i / (2 * N) / B;
  const SeqOut &to = m < N ? db : dc;
  if (!to.p) return;
  float s = 0.f;
  if (!lengths || t < lengths[b])
    for (int g = 0; g < groups; ++g) s += part[g * all + i];
  static_cast<T *>(to.p)[t * to.st + b * to.sb + m % N] = from_f<T>(s);
}

template <typename T, int LANES>
cudaError_t run(Args a, int *err, cudaStream_t s, int *launches) {
  const size_t bytes = shared_bytes<LANES>(a.warps);
  static PerDevice<cudaError_t> ready;
  const cudaError_t set = ready.here([] {
    return cudaFuncSetAttribute(scan_bwd_kernel<T, LANES>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)shared_bytes<LANES>(4));
  });
  if (set != cudaSuccess) return set;
  ++*launches;
  const int64_t blocks = (int64_t)a.groups * a.p.in.B * a.seg.n;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(32 * a.warps);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = s;
  return cudaLaunchKernelEx(&cfg, scan_bwd_kernel<T, LANES>, a, err);
}

}  // namespace

cudaError_t launch_scan_bwd(const ScanBwd &p, DevMem &ws, int *err, int nsm, bool vec,
                            cudaStream_t s, int *launches) {
  const ScanIn &in = p.in;
  const int64_t table = (int64_t)in.B * in.H * in.N, rows = (int64_t)in.B * in.H;
  Args a{};
  a.p = p;
  const int wc = 64 / lanes_of(in.N);
  a.warps = std::min(ceil_div(in.H, wc), lanes_of(in.N) == 1 ? 2 : 4);
  a.groups = ceil_div(in.H, wc * a.warps);
  a.seg = segments_of(in.T, (int64_t)a.groups * in.B, nsm, 3);
  const bool bc = p.db.p || p.dc.p, sums = p.da_log || p.dd || p.ddt_bias;
  const int64_t n_bc = bc ? (int64_t)a.groups * in.T * in.B * 2 * in.N : 0;
  const int64_t n_part = sums ? (int64_t)a.seg.n * in.B * in.H * (in.N + 2) : 0;
  const int64_t n_seg = a.seg.n > 1 ? a.seg.n * (table + rows) : 0;
  float *mem = nullptr;
  auto up = [](int64_t v) { return (v + 31) / 32 * 32; };
  if (n_bc + n_part + n_seg) {
    const cudaError_t e = ws.get((size_t)(up(n_bc) + up(n_part) + up(n_seg)) * 4, &mem);
    if (e != cudaSuccess) return e;
  }
  if (bc) a.part_bc = mem;
  if (sums) a.part = mem + up(n_bc);
  a.enter = p.dh_n;
  if (n_seg) {
    Meeting m{a.seg, mem + up(n_bc) + up(n_part), nullptr};
    m.sums = m.end + a.seg.n * table;
    const cudaError_t e = launch_local(in, true, p.dy, p.dh_n, m, err, vec, s, launches);
    if (e != cudaSuccess) return e;
    a.enter = m.end;
  }
  a.wide_states = vec && in.N % S == 0 && aligned(in.a_log, 4, 4, 4) && aligned(p.states, 4, 4, 4) &&
                  (!a.enter || aligned(a.enter, 4, 4, 4));
  cudaError_t e = by_lanes(in.N, [&](auto lanes) {
    constexpr int L = decltype(lanes)::value;
    return in.dtype == RCU_BF16 ? run<bf16, L>(a, err, s, launches) : run<float, L>(a, err, s, launches);
  });
  if (e != cudaSuccess) return e;
  if (sums) {
    const ColumnSum c{a.part, a.seg.n * (int64_t)in.B, (int64_t)in.H * (in.N + 2), (int64_t)in.H * in.N,
                      in.H, p.da_log, p.dd, p.ddt_bias};
    e = launch_column_sum(c, s, launches);
    if (e != cudaSuccess) return e;
  }
  if (bc) {
    const dim3 grid((unsigned)(((int64_t)in.T * in.B * 2 * in.N + 255) / 256));
    ++*launches;
    auto fn = in.dtype == RCU_BF16 ? sum_bc_kernel<bf16> : sum_bc_kernel<float>;
    e = launch_after(fn, grid, 256, s, (const float *)a.part_bc, a.groups, in.T, in.B, in.N, in.lengths,
                     p.db, p.dc);
  }
  return e;
}

}  // namespace rcu
