// Rotary positions: tables of (scaled) frequencies filled on the device, and the rotation of
// heads in both pair layouts over all or part of the head.
#include <cmath>

#include "rotary.cuh"

namespace qcf {

constexpr int kMaxRotaryPairs = 256;   // R <= 512
struct FreqTable {
  double w[kMaxRotaryPairs];
};

// One thread per table entry: the angle p w_k in fp64, its cosine and sine rounded once.
__global__ void __launch_bounds__(256) rope_table_kernel(float* __restrict__ cos_t, float* __restrict__ sin_t, int first_pos,
                                                         int64_t n, int half, double amplitude,
                                                         const __grid_constant__ FreqTable f) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (i >= n) return;
  const int64_t p = i / half;
  double s, c;
  sincos((static_cast<double>(first_pos) + static_cast<double>(p)) * f.w[i - p * half], &s, &c);
  cos_t[i] = static_cast<float>(c * amplitude);
  sin_t[i] = static_cast<float>(s * amplitude);
}

// One thread per (row, item, chunk of kRopeHeads heads): the angles of a row's item are read
// once and serve every head of the chunk, whose loads are all in flight together.
constexpr int kRopeHeads = 4;
template <typename T, int V>
__global__ void __launch_bounds__(256) rope_apply_kernel(const T* x, int64_t x_stride, T* y, int64_t y_stride, int n, int H,
                                                         int D, int R, const int32_t* __restrict__ pos,
                                                         const float* __restrict__ cos_t, const float* __restrict__ sin_t,
                                                         int max_pos, bool interleaved, bool inverse, unsigned int* status) {
  const int items = D / 2 / V, chunks = (H + kRopeHeads - 1) / kRopeHeads;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  const int64_t unit = t / items;
  const int item = static_cast<int>(t - unit * items);
  const int64_t row = unit / chunks;
  if (row >= n) return;
  const int h0 = static_cast<int>(unit - row * chunks) * kRopeHeads;
  const int p = pos[row];
  if (p < 0 || p >= max_pos) {
    if (p != -1 && h0 == 0 && item == 0) flag_status(status, QCF_DEV_BAD_INDEX);
    return;
  }
  const ItemAt at = item_at<V>(item, R, interleaved);
  const T* xr = x + row * x_stride;
  T* yr = y + row * y_stride;
  Vec<T, V> a[kRopeHeads], b[kRopeHeads];
#pragma unroll
  for (int i = 0; i < kRopeHeads; ++i)
    if (h0 + i < H) {
      a[i] = *reinterpret_cast<const Vec<T, V>*>(xr + (h0 + i) * D + at.a);
      b[i] = *reinterpret_cast<const Vec<T, V>*>(xr + (h0 + i) * D + at.b);
    }
  if (at.turns) {
    const Angles<V> g = load_angles<V>(cos_t, sin_t, p, R, item, inverse);
#pragma unroll
    for (int i = 0; i < kRopeHeads; ++i)
      if (h0 + i < H) turn_item<T, V>(a[i], b[i], g, interleaved);
  }
#pragma unroll
  for (int i = 0; i < kRopeHeads; ++i)
    if (h0 + i < H) {
      *reinterpret_cast<Vec<T, V>*>(yr + (h0 + i) * D + at.a) = a[i];
      *reinterpret_cast<Vec<T, V>*>(yr + (h0 + i) * D + at.b) = b[i];
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
  rope_apply_kernel<T, V><<<static_cast<unsigned>((threads + 255) / 256), 256, 0, r.st>>>(
      static_cast<const T*>(r.x), r.x_stride, static_cast<T*>(r.y), r.y_stride, r.n, r.H, r.D, r.R, r.pos, r.t->cos, r.t->sin,
      r.t->max_pos, (r.mode & QCF_ROPE_INTERLEAVED) != 0, (r.mode & QCF_ROPE_INVERSE) != 0, device_status_ptr());
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
  const int64_t n = static_cast<int64_t>(n_pos) * (R / 2);
  const int64_t blocks = (n + 255) / 256;
  if (blocks > INT32_MAX) return set_error(QCF_ERR_SHAPE, "qcf_rope_table_fill: %lld entries", (long long)n);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  LaunchScope ls(KC_ROPE_TABLE, st);
  rope_table_kernel<<<static_cast<unsigned>(blocks), 256, 0, st>>>(cos, sin, first_pos, n, R / 2, amplitude, f);
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
  if (static_cast<int64_t>(n) * ((H + kRopeHeads - 1) / kRopeHeads) * (D / 2) / 256 >= INT32_MAX)
    return set_error(QCF_ERR_SHAPE, "qcf_rope_apply: %d rows of %d x %d entries are too many for one call", n, H, D);
  if (n == 0) return QCF_OK;
  const RopeApply r{x, x_stride, y, y_stride, n, H, D, R, pos, t, mode, static_cast<cudaStream_t>(stream)};
  const cudaError_t e = dtype == QCF_BF16  ? rope_apply_type<__nv_bfloat16>(r)
                        : dtype == QCF_F16 ? rope_apply_type<__half>(r)
                                           : rope_apply_type<float>(r);
  return e == cudaSuccess ? QCF_OK : cuda_error(e, "qcf_rope_apply: launch");
}

}  // extern "C"
