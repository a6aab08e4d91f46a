// Rotary positions: tables of (scaled) frequencies filled on the device, and the rotation of
// heads in both pair layouts over all or part of the head.
#include <algorithm>
#include <cmath>

#include "rotary.cuh"

namespace qcf {

constexpr int kMaxRotaryPairs = 256;   // R <= 512
struct FreqTable {
  double w[kMaxRotaryPairs];
};

// Cosine and sine of p w as sums of two floats each (48 bits), and their product: angles add.
struct TwoSinCos {
  float c, cl, s, sl;
};
// a b - x y (SIGN = -1) or a b + x y (SIGN = +1) of two-float numbers: the leading products exactly
// (product and its rounding error), the cross terms to 32 bits, the leading sum with its error.
template <int SIGN>
__device__ __forceinline__ void two_dot(float ah, float al, float bh, float bl, float xh, float xl, float yh, float yl, float& sum,
                                        float& rest) {
  const float xs = SIGN * xh, xls = SIGN * xl;
  const float p = __fmul_rn(ah, bh), q = __fmul_rn(xs, yh);
  float lo = __fadd_rn(__fmaf_rn(ah, bh, -p), __fmaf_rn(xs, yh, -q));
  lo = __fmaf_rn(ah, bl, lo);
  lo = __fmaf_rn(al, bh, lo);
  lo = __fmaf_rn(xs, yl, lo);
  lo = __fmaf_rn(xls, yh, lo);
  sum = __fadd_rn(p, q);
  const float t = __fsub_rn(sum, p);
  rest = __fadd_rn(__fadd_rn(__fsub_rn(p, __fsub_rn(sum, t)), __fsub_rn(q, t)), lo);
}
__device__ __forceinline__ TwoSinCos two_add(const TwoSinCos& a, const TwoSinCos& b) {
  float h, l;
  TwoSinCos r;
  two_dot<-1>(a.c, a.cl, b.c, b.cl, a.s, a.sl, b.s, b.sl, h, l);
  r.c = __fadd_rn(h, l);
  r.cl = __fsub_rn(l, __fsub_rn(r.c, h));
  two_dot<1>(a.s, a.sl, b.c, b.cl, a.c, a.cl, b.s, b.sl, h, l);
  r.s = __fadd_rn(h, l);
  r.sl = __fsub_rn(l, __fsub_rn(r.s, h));
  return r;
}

// Table entries of PAIRS pairs (blockIdx.y) and na blocks of 256 positions (blockIdx.x).  fp64 runs
// at 1/64 of the fp32 rate here: a sine and cosine in fp64 of every entry took 511 us for 131072
// positions of 64 pairs, 50 times the write.  Instead a position is taken apart in base 4,
// p = 256 a + 64 b1 + 16 b0 + 4 c1 + c0; the fp64 values of the na + 12 parts of a pair become
// two-float numbers, their angles are added in those (four additions, 2^-47 each), and each entry
// is rounded once.  The parts are of the position itself, so an entry's bits do not depend on the
// call that fills it.  Thread = (pair, b and part of c): it forms b + c once and uses it for every a,
// and a warp writes runs of 4 PAIRS bytes.  1024 threads: one CTA per SM has the fewest fp64 values.
// 131072 positions of 64 pairs, 16 to a CTA: 23 us, 2.9 TB/s.  About 16 of them are the additions and stores:
// without the fp64 values the kernel takes 18.3, and one that returns behind them 6.2, launch
// included (32, whole 128-byte lines but twice the fp64 values per SM: 28 us).  8192 positions of 32 pairs: 5.7 us with 8 to a CTA, 8.5 with 16,
// which fills 64 SMs only.
constexpr int kTableThreads = 1024;
template <int PAIRS>
__global__ void __launch_bounds__(kTableThreads) rope_table_kernel(float* __restrict__ cos_t, float* __restrict__ sin_t, int first_pos,
                                                                   int n_pos, int half, int na, double amplitude,
                                                                   const __grid_constant__ FreqTable f) {
  constexpr int PER = 256 * PAIRS / kTableThreads;   // positions of a thread in each block
  __shared__ TwoSinCos a_s[16][PAIRS], digit[4][4][PAIRS];
  const int k0 = blockIdx.y * PAIRS;
  const int64_t a0 = first_pos / 256 + static_cast<int64_t>(blockIdx.x) * na;
  for (int e = threadIdx.x; e < (na + 12) * PAIRS; e += kTableThreads) {
    const int i = e / PAIRS, k = e % PAIRS;
    if (k0 + k >= half) continue;
    const int j = i - na;   // digit j % 3 + 1 of place j / 3
    const double mult = j < 0 ? 256.0 * static_cast<double>(a0 + i) : static_cast<double>((j % 3 + 1) << (2 * (j / 3)));
    double s, c;
    sincos(mult * f.w[k0 + k], &s, &c);
    if (j < 0) {
      s *= amplitude;
      c *= amplitude;
    }
    TwoSinCos v;
    v.c = static_cast<float>(c);
    v.cl = static_cast<float>(c - v.c);
    v.s = static_cast<float>(s);
    v.sl = static_cast<float>(s - v.s);
    (j < 0 ? a_s[i] : digit[j / 3][j % 3 + 1])[k] = v;
  }
  if (threadIdx.x < 4 * PAIRS) digit[threadIdx.x / PAIRS][0][threadIdx.x % PAIRS] = TwoSinCos{1.f, 0.f, 0.f, 0.f};
  __syncthreads();
  const int k = threadIdx.x % PAIRS;
  if (k0 + k >= half) return;
  const int64_t step = static_cast<int64_t>(256) * half;
  for (int c = 0; c < PER; ++c) {
    const int p = threadIdx.x / PAIRS * PER + c;
    const TwoSinCos d = two_add(two_add(digit[3][p >> 6][k], digit[2][p >> 4 & 3][k]),
                                two_add(digit[1][p >> 2 & 3][k], digit[0][p & 3][k]));
    const int64_t row = 256 * a0 + p - first_pos;   // of a = 0; the table holds rows 0 .. n_pos - 1
    const int a_lo = row < 0 ? 1 : 0;               // the first block may begin before first_pos
    const int64_t left = row < n_pos ? (n_pos - 1 - row) / 256 + 1 : 0;
    const int a_hi = left < na ? static_cast<int>(left) : na;
    float* cr = cos_t + (row + 256 * a_lo) * half + k0 + k;
    float* sr = sin_t + (row + 256 * a_lo) * half + k0 + k;
#pragma unroll 4
    for (int a = a_lo; a < a_hi; ++a, cr += step, sr += step) {
      const TwoSinCos v = a_s[a][k];
      float h, l;
      two_dot<-1>(v.c, v.cl, d.c, d.cl, v.s, v.sl, d.s, d.sl, h, l);
      *cr = __fadd_rn(h, l);
      two_dot<1>(v.s, v.sl, d.c, d.cl, v.c, v.cl, d.s, d.sl, h, l);
      *sr = __fadd_rn(h, l);
    }
  }
}

// One thread per (row, item, chunk of kRopeHeads heads): the angles of a row's item are read
// once and serve every head of the chunk, whose loads are all in flight together (and before the
// position is known).  HBM-bound: 17984 rows of 72 heads of 128 in bf16 take 97.7 us, 6.8 TB/s, the
// rate of a copy; with the entries unpacked as they come (twice the registers) 152 us, with 8 heads
// to a thread 224.  In fp32 eight pairs of four heads are 64 registers of entries: the kernel spills 144
// bytes a thread and takes 210 us for the same rows (floor 195), neighbours 246.  Runs shorter than 8
// move fewer bytes an access: heads of 80 turned whole 65 us (floor 61), 32 of the 80 entries 68, 20 of them 75.
constexpr int kRopeHeads = 4;
template <typename T, int V, bool INTER>
__global__ void __launch_bounds__(256, 3) rope_apply_kernel(const T* x, int64_t x_stride, T* y, int64_t y_stride, int n, int H,
                                                         int D, int R, const int32_t* __restrict__ pos,
                                                         const float* __restrict__ cos_t, const float* __restrict__ sin_t,
                                                         int max_pos, bool inverse, unsigned int* status) {
  const unsigned items = D / 2 / V, chunks = (H + kRopeHeads - 1) / kRopeHeads;
  const unsigned t = blockIdx.x * 256u + threadIdx.x;
  const unsigned unit = t / items, item = t - unit * items, row = unit / chunks;
  if (row >= static_cast<unsigned>(n)) return;
  const int h0 = static_cast<int>(unit - row * chunks) * kRopeHeads;
  const ItemAt at = item_at<V, INTER>(item, R);
  const T* xr = x + row * x_stride;
  T* yr = y + row * y_stride;
  const int p = pos[row];
  Run<T, V> a[kRopeHeads], b[kRopeHeads];
#pragma unroll
  for (int i = 0; i < kRopeHeads; ++i)
    if (h0 + i < H) {
      a[i].load(xr + (h0 + i) * D + at.a);
      b[i].load(xr + (h0 + i) * D + at.b);
    }
  if (p < 0 || p >= max_pos) {
    if (p != -1 && h0 == 0 && item == 0) flag_status(status, QCF_DEV_BAD_INDEX);
    return;
  }
  if (at.turns) {
    const Angles<V> g = load_angles<V>(cos_t, sin_t, p, R, item, inverse);
#pragma unroll
    for (int i = 0; i < kRopeHeads; ++i)
      if (h0 + i < H) turn_item<T, V, INTER>(a[i], b[i], g);
  }
#pragma unroll
  for (int i = 0; i < kRopeHeads; ++i)
    if (h0 + i < H) {
      a[i].store(yr + (h0 + i) * D + at.a);
      b[i].store(yr + (h0 + i) * D + at.b);
    }
}

struct RopeApply {
  const void* x;
  int64_t x_stride;
  void* y;
  int64_t y_stride;
  int n, H, D, R;
  const int32_t* pos;
  const qcf_rope_table* t;
  int mode;
  cudaStream_t st;
};

template <typename T, int V>
static cudaError_t rope_apply_launch(const RopeApply& r) {
  const int64_t threads = static_cast<int64_t>(r.n) * ((r.H + kRopeHeads - 1) / kRopeHeads) * (r.D / 2 / V);
  LaunchScope ls(KC_ROPE_APPLY, r.st);
  const auto kernel = r.mode & QCF_ROPE_INTERLEAVED ? rope_apply_kernel<T, V, true> : rope_apply_kernel<T, V, false>;
  kernel<<<static_cast<unsigned>((threads + 255) / 256), 256, 0, r.st>>>(
      static_cast<const T*>(r.x), r.x_stride, static_cast<T*>(r.y), r.y_stride, r.n, r.H, r.D, r.R, r.pos, r.t->cos, r.t->sin,
      r.t->max_pos, (r.mode & QCF_ROPE_INVERSE) != 0, device_status_ptr());
  return cudaGetLastError();
}

template <typename T>
static cudaError_t rope_apply_type(const RopeApply& r) {
  switch (item_width(r.R, r.D, r.x_stride, r.y_stride)) {
    case 8: return rope_apply_launch<T, 8>(r);
    case 4: return rope_apply_launch<T, 4>(r);
    case 2: return rope_apply_launch<T, 2>(r);
    default: return rope_apply_launch<T, 1>(r);
  }
}

// Frequencies of one table: theta^(-2k/R), scaled as the header describes.
static qcf_status rope_frequencies(int R, double theta, const qcf_rope_scaling* sc, FreqTable* f, double* amplitude) {
  const char* who = "qcf_rope_table_fill";
  const int half = R / 2;
  const int kind = sc ? sc->kind : QCF_ROPE_SCALE_NONE;
  if (kind < QCF_ROPE_SCALE_NONE || kind > QCF_ROPE_SCALE_INDEX)
    return set_error(QCF_ERR_INVALID_ARG, "%s: unknown scaling kind %d", who, kind);
  *amplitude = sc ? sc->amplitude : 1.0;
  if (!std::isfinite(*amplitude)) return set_error(QCF_ERR_INVALID_ARG, "%s: amplitude is not finite", who);
  if (kind != QCF_ROPE_SCALE_NONE && !(sc->factor >= 1.0 && std::isfinite(sc->factor)))
    return set_error(QCF_ERR_INVALID_ARG, "%s: factor %g below 1", who, sc->factor);
  if (kind >= QCF_ROPE_SCALE_TURNS) {
    const bool ok = sc->original > 0 && sc->low < sc->high && std::isfinite(sc->high) &&
                    (kind == QCF_ROPE_SCALE_TURNS ? sc->low >= 0.0 : sc->low > 0.0);
    if (!ok)
      return set_error(QCF_ERR_INVALID_ARG, "%s: original=%d low=%g high=%g", who, sc->original, sc->low, sc->high);
  }
  if (kind == QCF_ROPE_SCALE_BASE) {
    if (R <= 2) return set_error(QCF_ERR_SHAPE, "%s: base scaling needs R > 2", who);
    theta *= std::pow(sc->factor, static_cast<double>(R) / (R - 2));
  }
  const double pi = 3.14159265358979323846;
  double a = 0, b = 0;
  if (kind == QCF_ROPE_SCALE_INDEX) {
    auto index_of = [&](double turns) { return R * std::log(sc->original / (2 * pi * turns)) / (2 * std::log(theta)); };
    a = std::max(0.0, std::floor(index_of(sc->high)));
    b = std::min(half - 1.0, std::ceil(index_of(sc->low)));
  }
  for (int k = 0; k < half; ++k) {
    double w = std::pow(theta, -2.0 * k / R);
    if (kind == QCF_ROPE_SCALE_LINEAR) w /= sc->factor;
    if (kind >= QCF_ROPE_SCALE_TURNS) {
      double g = kind == QCF_ROPE_SCALE_TURNS ? (sc->original * w / (2 * pi) - sc->low) / (sc->high - sc->low)
                                              : 1.0 - (k - a) / std::max(b - a, 1e-3);
      g = std::min(1.0, std::max(0.0, g));
      w *= g + (1.0 - g) / sc->factor;
    }
    f->w[k] = w;
  }
  return QCF_OK;
}

}  // namespace qcf

using namespace qcf;

extern "C" {

qcf_status qcf_rope_table_fill(float* cos, float* sin, int first_pos, int n_pos, int R, double theta,
                               const qcf_rope_scaling* scaling, void* stream) {
  if (!cos || !sin) return set_error(QCF_ERR_INVALID_ARG, "qcf_rope_table_fill: NULL pointer");
  if (!(theta > 1.0) || !std::isfinite(theta)) return set_error(QCF_ERR_INVALID_ARG, "qcf_rope_table_fill: theta=%g", theta);
  if (first_pos < 0 || n_pos < 0 || first_pos > INT32_MAX - n_pos || R < 2 || (R & 1) || R > 2 * kMaxRotaryPairs)
    return set_error(QCF_ERR_SHAPE, "qcf_rope_table_fill: first_pos=%d n_pos=%d R=%d", first_pos, n_pos, R);
  if (take_fault(4) || !aligned16(cos) || !aligned16(sin))
    return set_error(QCF_ERR_ALIGN, "qcf_rope_table_fill: tables must be 16-byte aligned");
  FreqTable f;
  double amplitude;
  const qcf_status s = rope_frequencies(R, theta, scaling, &f, &amplitude);
  if (s != QCF_OK) return s;
  if (n_pos == 0) return QCF_OK;
  // blocks of 256 positions, up to 16 to a CTA, so that one CTA per SM does; 16 pairs to a CTA, or 8
  // where that leaves SMs idle (its fp64 values are then most of the time)
  const int64_t blocks = (static_cast<int64_t>(first_pos) + n_pos + 255) / 256 - first_pos / 256;
  const bool few = blocks * ((R / 2 + 15) / 16) < num_sms();
  const int groups = few ? (R / 2 + 7) / 8 : (R / 2 + 15) / 16;
  const int na = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(16, (blocks * groups + num_sms() - 1) / num_sms())));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  LaunchScope ls(KC_ROPE_TABLE, st);
  const auto kernel = few ? rope_table_kernel<8> : rope_table_kernel<16>;
  kernel<<<dim3(static_cast<unsigned>((blocks + na - 1) / na), groups), kTableThreads, 0, st>>>(cos, sin, first_pos, n_pos, R / 2, na,
                                                                                           amplitude, f);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? QCF_OK : cuda_error(e, "qcf_rope_table_fill: launch");
}

qcf_status qcf_rope_apply(const void* x, int64_t x_stride, void* y, int64_t y_stride, int n, int H, int D, int dtype,
                          const int32_t* pos, const qcf_rope_table* t, int mode, void* stream) {
  if (!x || !y || !pos || !t || !t->cos || !t->sin) return set_error(QCF_ERR_INVALID_ARG, "qcf_rope_apply: NULL pointer");
  if (dtype < QCF_BF16 || dtype > QCF_F32 || (mode & ~(QCF_ROPE_INTERLEAVED | QCF_ROPE_INVERSE)))
    return set_error(QCF_ERR_INVALID_ARG, "qcf_rope_apply: dtype=%d mode=%d", dtype, mode);
  const int R = t->head_dim;
  if (n < 0 || H <= 0 || H > 65535 || D < 2 || (D & 1) || D > 512 || R < 2 || (R & 1) || R > D || t->max_pos <= 0)
    return set_error(QCF_ERR_SHAPE, "qcf_rope_apply: n=%d H=%d D=%d rotated width %d", n, H, D, R);
  if (x_stride < static_cast<int64_t>(H) * D || y_stride < static_cast<int64_t>(H) * D || (x == y && x_stride != y_stride))
    return set_error(QCF_ERR_SHAPE, "qcf_rope_apply: row strides %lld, %lld for %d x %d entries", (long long)x_stride,
                     (long long)y_stride, H, D);
  if (take_fault(4) || !aligned16(x) || !aligned16(y) || !aligned16(t->cos) || !aligned16(t->sin))
    return set_error(QCF_ERR_ALIGN, "qcf_rope_apply: pointers must be 16-byte aligned");
  if (take_fault(1)) return set_error(QCF_ERR_INVALID_ARG, "qcf_rope_apply: injected invalid index table");
  // threads are counted in 32 bits
  if (static_cast<int64_t>(n) * ((H + kRopeHeads - 1) / kRopeHeads) * (D / 2 / item_width(R, D, x_stride, y_stride)) > UINT32_MAX - 256)
    return set_error(QCF_ERR_SHAPE, "qcf_rope_apply: %d rows of %d x %d entries are too many for one call", n, H, D);
  if (n == 0) return QCF_OK;
  const RopeApply r{x, x_stride, y, y_stride, n, H, D, R, pos, t, mode, static_cast<cudaStream_t>(stream)};
  const cudaError_t e = dtype == QCF_BF16  ? rope_apply_type<__nv_bfloat16>(r)
                        : dtype == QCF_F16 ? rope_apply_type<__half>(r)
                                           : rope_apply_type<float>(r);
  return e == cudaSuccess ? QCF_OK : cuda_error(e, "qcf_rope_apply: launch");
}

}  // extern "C"
