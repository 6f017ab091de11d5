// The experts' products: rows in expert order times the matrix of their expert, and the gradients.
//
// With R_e the rows of expert e, X their inputs, Y their outputs and W_e its matrix,
//     Y = X W_e,   dX = dY W_e',   dW_e = X' dY     (R_e x inputs x outputs each).
// All three are C = A B for every expert: in the first two the rows are a size of C (ragged), in the third they are
// what is summed over.  How many rows an expert has is known on the device only, so a workgroup finds its
// expert and rows from the offsets: tiles are counted through the experts in order, one wave's lanes a
// few experts each.
#include "hard_dev.hpp"
#include "hard_internal.hpp"

namespace lapsum {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));

LDEV f32x4 mfma(pack_t<bf16> a, pack_t<bf16> b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
LDEV f32x4 mfma(pack_t<f16> a, pack_t<f16> b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

LDEV int offset_of(const ProductArgs &p, int i) {
  const int64_t o = p.offsets[i];
  return (int)(o < 0 ? 0 : (o > p.rows ? p.rows : o));
}

// The rows in order are those before the first expert's, every expert's, and those behind the
// last one's: experts + 2 ranges, of which the first and the last are no expert's.
LDEV int range_begin(const ProductArgs &p, int g) {
  return g == 0 ? 0 : (g <= p.experts + 1 ? offset_of(p, g - 1) : (int)p.rows);
}

struct RowTile {
  int expert;      // -1: no expert's
  int first, end;  // rows of the tile
};
// The index-th of the tiles of `size` rows; every wave finds it by itself.  False: there are no more.
LDEV bool find_rows(const ProductArgs &p, int size, int index, RowTile &t) {
  const int lane = lane_id(), ranges = p.experts + 2, per = (ranges + 63) / 64;
  int mine = 0;
  for (int i = 0; i < per; ++i) {
    const int g = lane * per + i;
    if (g >= ranges) break;
    const int a = range_begin(p, g), b = range_begin(p, g + 1);
    mine += b > a ? (b - a + size - 1) / size : 0;
  }
  int upto = mine;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int x = __shfl_up(upto, d, 64);
    if (lane >= d) upto += x;
  }
  if (index >= read_lane(upto, 63)) return false;
  const int at = __builtin_ctzll(__ballot(upto > index));
  int left = index - read_lane(upto - mine, at);
  for (int i = 0; i < per; ++i) {
    const int g = at * per + i;
    if (g >= ranges) break;
    const int a = range_begin(p, g), b = range_begin(p, g + 1), n = b > a ? (b - a + size - 1) / size : 0;
    if (left < n) {
      t.expert = g >= 1 && g <= p.experts ? g - 1 : -1;
      t.first = a + left * size;
      t.end = t.first + size < b ? t.first + size : b;
      return true;
    }
    left -= n;
  }
  return false;
}
// as many tiles as there can be
int64_t most_row_tiles(const ProductArgs &p, int size) { return p.rows / size + p.experts + 2; }

// ------------------------------------------------------------------ any layout
// A tile of 64 x 64, its factors brought to LDS an element at a time: for sizes, strides and pointers that are no
// multiples of 16 bytes.
constexpr int kAny = 64, kAnyK = 32;

template <class T, bool SUM_ROWS>
__global__ __launch_bounds__(256) void product_any_kernel(ProductArgs p) {
  __shared__ struct {
    T a[kAny][kAnyK + 8], b[kAny][kAnyK + 8];
  } sh;
  lds_poison(sh);
  const int n0 = blockIdx.x * kAny;
  int m0, m1, k0, k1, e;
  if (SUM_ROWS) {
    const int tiles = (p.m + kAny - 1) / kAny;
    if (grid_row() >= (int64_t)tiles * p.experts) return;
    e = (int)(grid_row() / tiles);
    m0 = (int)(grid_row() % tiles) * kAny;
    m1 = m0 + kAny < p.m ? m0 + kAny : p.m;
    k0 = offset_of(p, e);
    k1 = offset_of(p, e + 1);
  } else {
    RowTile t;
    if (grid_row() > 0x7FFFFFFF || !find_rows(p, kAny, (int)grid_row(), t)) return;
    e = t.expert;
    m0 = t.first;
    m1 = t.end;
    k0 = 0;
    k1 = e < 0 ? 0 : p.k;
  }
  const T *a = static_cast<const T *>(p.a), *b = static_cast<const T *>(p.b);
  if (!SUM_ROWS && e >= 0) b += e * p.be;
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64, i = threadIdx.x;
  f32x4 c[4] = {};
  for (int k = k0; k < k1; k += kAnyK) {
    // neighbouring lanes take neighbouring elements where there are any
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int x = j * 256 + i, at = p.ak == 1 ? x / kAnyK : x % kAny, kk = p.ak == 1 ? x % kAnyK : x / kAny;
      const bool there = m0 + at < m1 && k + kk < k1;
      sh.a[at][kk] = there ? a[(m0 + at) * p.am + (k + kk) * p.ak] : (T)0.0f;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int x = j * 256 + i, at = p.bk == 1 ? x / kAnyK : x % kAny, kk = p.bk == 1 ? x % kAnyK : x / kAny;
      const bool there = n0 + at < p.n && k + kk < k1;
      sh.b[at][kk] = there ? b[(n0 + at) * p.bn + (k + kk) * p.bk] : (T)0.0f;
    }
    __syncthreads();
    const pack_t<T> f = load_pack(&sh.a[wave * 16 + lane % 16][lane / 16 * 8]);
#pragma unroll
    for (int j = 0; j < 4; ++j) c[j] = mfma(f, load_pack(&sh.b[j * 16 + lane % 16][lane / 16 * 8]), c[j]);
    __syncthreads();
  }
  T *out = static_cast<T *>(p.c) + (SUM_ROWS ? e * p.ce : 0);
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int m = m0 + wave * 16 + lane / 16 * 4 + r;
    if (m >= m1) continue;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int n = n0 + j * 16 + lane % 16;
      if (n < p.n) out[m * p.cm + n] = (T)c[j][r];
    }
  }
}

template <class T>
hipError_t rows_of(const ProductArgs &p, hipStream_t s) {
  const unsigned nt = (unsigned)((p.n + kAny - 1) / kAny);
  product_any_kernel<T, false><<<rows_grid(nt, most_row_tiles(p, kAny)), dim3(256), 0, s>>>(p);
  return hipGetLastError();
}
template <class T>
hipError_t weights_of(const ProductArgs &p, hipStream_t s) {
  const unsigned nt = (unsigned)((p.n + kAny - 1) / kAny);
  const int64_t mt = (p.m + kAny - 1) / kAny;
  product_any_kernel<T, true><<<rows_grid(nt, mt * p.experts), dim3(256), 0, s>>>(p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_product_rows(const ProductArgs &p, int dtype, hipStream_t s) {
  return dtype == LAPSUM_BF16 ? rows_of<bf16>(p, s) : rows_of<f16>(p, s);
}
hipError_t launch_product_weights(const ProductArgs &p, int dtype, hipStream_t s) {
  return dtype == LAPSUM_BF16 ? weights_of<bf16>(p, s) : weights_of<f16>(p, s);
}

}  // namespace lapsum
