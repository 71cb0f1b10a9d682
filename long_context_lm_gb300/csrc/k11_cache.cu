// k11_cache.cu -- writing rows into the paged cache (fs_cache_append), reading
// them back (fs_cache_read) and moving the rows of an accepted path
// (fs_cache_accept).
//
// A row of d elements belongs to d / 16 neighbouring lanes, sixteen elements (two
// 16-byte pieces of bf16) each; the row's largest magnitude is a shuffle
// reduction over them.  A block takes up to 256 tokens of one (sequence, head,
// key or value); their pages are looked up once, into shared memory, and all
// loads of a thread stand before their first use.  Bound by memory (append: 2 d
// bytes in, d bits / 8 + 4 out a row; read: the other way) as long as no more
// than some ten instructions an element are spent: with eight elements a lane and
// a page lookup a row, append was bound by instructions (65536 x 16 x 64 bf16 to
// e4m3: 113 us).
//
// Codes without a division an element.  q = Q x / amax is a fraction of small
// integers: with x = X 2^f, amax = A 2^e (X, A < 2^8) and a border between two
// codes m = M 2^g (M < 2^8), q = m or |q - m| >= 2^-16 m: the difference of
// Q X 2^(f-e) and A M 2^g is a multiple of the smaller unit.  x * fl(Q / amax)
// is within 2^-22 of q.  Rounded to 18 significant bits it is m exactly if q
// is, and on the same side of m as q otherwise; then the one rounding to a code,
// ties to even, decides as for q itself.
#include "cache.cuh"

namespace fs {
namespace {

constexpr uint32_t kInfBits = 0x7f800000u;

// Q x / amax to 18 significant bits, s = Q / amax.
__device__ __forceinline__ float quotient(float x, float s) {
  return __uint_as_float((__float_as_uint(x * s) + 0x20u) & ~0x3fu);
}
// Nearest integer, ties to even, in the low bits.
__device__ __forceinline__ uint32_t nearest(float q) { return __float_as_uint(q + 12582912.f); }

// Code words of a lane's sixteen elements: 8, 4 or 2.
template <int F>
constexpr int kWords = Fmt<F>::kBits / 2;

template <int F>
__device__ __forceinline__ void encode(const uint32_t (&x)[8], float amax, uint32_t (&w)[8]) {
  if constexpr (F == FS_CACHE_BF16) {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = x[i];
  } else {
#pragma unroll
    for (int i = 0; i < kWords<F>; ++i) w[i] = 0;
    if (!(amax > 0.f) || !(amax < __uint_as_float(kInfBits))) return;
    float v[16];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[2 * i] = bf16_lo(x[i]);
      v[2 * i + 1] = bf16_hi(x[i]);
    }
    if (amax < 0x1p-64f) {  // Q / amax must not pass the fp32 range
      amax *= 0x1p64f;
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] *= 0x1p64f;
    }
    const float s = __fdiv_rn(Fmt<F>::kTop, amax);
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = quotient(v[i], s);
#pragma unroll
    for (int i = 0; i < kWords<F>; ++i) {
      if constexpr (F == FS_CACHE_E4M3) {
        asm("{\n .reg .b16 lo, hi;\n cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n"
            " cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n mov.b32 %0, {lo, hi};\n}\n"
            : "=r"(w[i])
            : "f"(v[4 * i]), "f"(v[4 * i + 1]), "f"(v[4 * i + 2]), "f"(v[4 * i + 3]));
      } else if constexpr (F == FS_CACHE_INT8) {
        w[i] = __byte_perm(__byte_perm(nearest(v[4 * i]), nearest(v[4 * i + 1]), 0x0040),
                           __byte_perm(nearest(v[4 * i + 2]), nearest(v[4 * i + 3]), 0x0040), 0x5410);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) w[i] |= (nearest(v[8 * i + j]) & 15u) << (4 * j);
      }
    }
  }
}

// N words to or from an address that is aligned to them, up to 16 bytes.
template <int N>
__device__ __forceinline__ void store_words(void *p, const uint32_t *w) {
  if constexpr (N == 2) {
    *static_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
  } else {
#pragma unroll
    for (int i = 0; i < N / 4; ++i)
      static_cast<uint4 *>(p)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
  }
}
template <int N>
__device__ __forceinline__ void load_words(const void *p, uint32_t *w) {
  if constexpr (N == 2) {
    const uint2 u = *static_cast<const uint2 *>(p);
    w[0] = u.x, w[1] = u.y;
  } else {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const uint4 u = static_cast<const uint4 *>(p)[i];
      w[4 * i] = u.x, w[4 * i + 1] = u.y, w[4 * i + 2] = u.z, w[4 * i + 3] = u.w;
    }
  }
}

// The tokens of a block and where they lie.
template <int L, int N>
struct Rows {
  static constexpr int kPass = 256 / L, kAll = kPass * N;
  static constexpr int kPages = kAll / 16 + 1;  // that kAll tokens can touch
  int b, h, part, lane, first, n;  // first token of the block; tokens of the sequence
  long long start;
  size_t base;  // row of head h, part, in page 0
  int shift;

  // False: the block has no token.
  __device__ __forceinline__ bool init(const CacheRowsArgs &a, int *pages) {
    b = blockIdx.y / a.c.Hkv;
    h = blockIdx.y - b * a.c.Hkv;
    part = blockIdx.z;
    lane = threadIdx.x % L;
    first = blockIdx.x * kAll;
    n = a.count ? min(a.count[b], a.T) : a.T;
    if (first >= n) return false;
    start = a.start[b];
    shift = 31 - __clz(a.c.page);
    base = cache_row(a.c, 0, part, h, 0);
    // pages of the block's tokens, by the first position in each; a position
    // before 0 has none
    const long long p0 = (start + first) >> shift;
    if (threadIdx.x < kPages) {
      const long long p = p0 + threadIdx.x;
      const int last = min(first + kAll, n) - 1;
      int page = -1, off;
      if (p <= (start + last) >> shift) page = cache_page(a.c, b, p << shift, &off);
      pages[threadIdx.x] = page;
    }
    __syncthreads();
    return true;
  }
  // Row of token first + i in the cache, or -1.
  __device__ __forceinline__ long long row(const CacheRowsArgs &a, const int *pages, int i) const {
    if (first + i >= n) return -1;
    const long long pos = start + first + i;
    const int page = pages[(int)((pos >> shift) - ((start + first) >> shift))];
    if (page < 0) return -1;
    return (long long)(base + (size_t)page * (2 * (size_t)a.c.Hkv << shift)) +
           (int)(pos & (a.c.page - 1));
  }
};

// Whole groups of lanes take part or not, and every lane reaches the shuffles.
template <int F, int L, int N>
__global__ void __launch_bounds__(256) k11_append_kernel(const __grid_constant__ CacheRowsArgs a) {
  using R = Rows<L, N>;
  __shared__ int pages[R::kPages];
  R r;
  if (!r.init(a, pages)) return;
  const long long(&s)[3] = r.part ? a.vs : a.ks;
  const uint16_t *p = static_cast<const uint16_t *>(r.part ? a.v : a.k) + r.b * s[0] + r.h * s[1] +
                      r.first * s[2] + r.lane * 16;
  uint32_t x[N][8];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int t = threadIdx.x / L + i * R::kPass;
#pragma unroll
    for (int j = 0; j < 8; ++j) x[i][j] = 0;
    if (r.first + t < r.n) load_words<8>(p + t * s[2], x[i]);
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float amax = 0.f;
    if constexpr (F != FS_CACHE_BF16) {
      // Magnitudes of bf16 compare as integers, NaN above infinity.
      uint32_t m = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) m = __vmaxu2(m, x[i][j] & 0x7fff7fffu);
#pragma unroll
      for (int o = L / 2; o > 0; o >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
      amax = __uint_as_float(max(m << 16, m & 0xffff0000u));
    }
    const long long row = r.row(a, pages, threadIdx.x / L + i * R::kPass);
    if (row < 0) continue;
    uint32_t w[8];
    encode<F>(x[i], amax, w);
    store_words<kWords<F>>(static_cast<char *>(a.c.codes) + (row * L + r.lane) * (4 * kWords<F>), w);
    if constexpr (F != FS_CACHE_BF16) {
      if (r.lane == 0)
        a.c.scales[row] = amax < __uint_as_float(kInfBits) ? __fdiv_rn(amax, Fmt<F>::kTop)
                                                           : __uint_as_float(0x7fc00000u);
    }
  }
}

template <int F, int L, int N, bool F32>
__global__ void __launch_bounds__(256) k11_read_kernel(const __grid_constant__ CacheRowsArgs a) {
  using R = Rows<L, N>;
  __shared__ int pages[R::kPages];
  R r;
  if (!r.init(a, pages)) return;
  uint32_t w[N][8];
  float s[N];
  bool have[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const long long row = r.row(a, pages, threadIdx.x / L + i * R::kPass);
    have[i] = row >= 0;
    s[i] = 1.f;
    if (have[i]) {
      load_words<kWords<F>>(
          static_cast<const char *>(a.c.codes) + (row * L + r.lane) * (4 * kWords<F>), w[i]);
      if constexpr (F != FS_CACHE_BF16) s[i] = a.c.scales[row];
    }
  }
  void *out = r.part ? a.v_out : a.k_out;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if (!have[i]) continue;
    const int t = r.first + threadIdx.x / L + i * R::kPass;
    const size_t at = (((size_t)blockIdx.y * a.T + t) * L + r.lane) * 16;
    if constexpr (F == FS_CACHE_BF16 && !F32) {
      store_words<8>(static_cast<uint16_t *>(out) + at, w[i]);
    } else {
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        float x[8];
        uint32_t c[4];
#pragma unroll
        for (int j = 0; j < kWords<F> / 2; ++j) c[j] = w[i][half * (kWords<F> / 2) + j];
        decode8<F>(c, x);
        if constexpr (F != FS_CACHE_BF16) {
#pragma unroll
          for (int j = 0; j < 8; ++j) x[j] *= s[i];
        }
        uint32_t y[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = F32 ? __float_as_uint(x[j]) : 0;
        if constexpr (F32) {
          store_words<8>(static_cast<float *>(out) + at + 8 * half, y);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) y[j] = pack_bf16(x[2 * j], x[2 * j + 1]);
          store_words<4>(static_cast<uint16_t *>(out) + at + 8 * half, y);
        }
      }
    }
  }
}

// One block per (sequence, kv head, part); a thread takes 16-byte pieces (at
// most 64 rows of 16 pieces), all read before the barrier and written after it.
__global__ void __launch_bounds__(256) k11_accept_kernel(const __grid_constant__ CacheRowsArgs a,
                                                         int words) {
  const int part = blockIdx.z, b = blockIdx.y / a.c.Hkv, h = blockIdx.y - b * a.c.Hkv;
  const int n = a.count ? min(a.count[b], a.T) : a.T;
  uint4 *codes = static_cast<uint4 *>(a.c.codes);
  uint4 x[4];
  float scale[4];
  long long to[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int item = threadIdx.x + i * blockDim.x, row = item / words, piece = item - row * words;
    to[i] = -1;
    if (row >= n) continue;
    const int from = a.path[(size_t)b * a.T + row];
    if (from < 0 || from >= 64) {
      if (a.c.status) atomicCAS(a.c.status, 0, FS_ERR_CACHE);
      continue;
    }
    int src_off, dst_off;
    const int src = cache_page(a.c, b, (long long)a.start[b] + from, &src_off);
    const int dst = cache_page(a.c, b, (long long)a.start[b] + row, &dst_off);
    if (src < 0 || dst < 0) continue;
    const size_t index = cache_row(a.c, src, part, h, src_off);
    x[i] = codes[index * words + piece];
    if (piece == 0 && a.c.format != FS_CACHE_BF16) scale[i] = a.c.scales[index];
    to[i] = (long long)cache_row(a.c, dst, part, h, dst_off);
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (to[i] < 0) continue;
    const int item = threadIdx.x + i * blockDim.x, piece = item % words;
    codes[(size_t)to[i] * words + piece] = x[i];
    if (piece == 0 && a.c.format != FS_CACHE_BF16) a.c.scales[to[i]] = scale[i];
  }
}

// Blocks along the tokens, (sequence, head), part.
template <int L, int N>
dim3 row_grid(const CacheRowsArgs &a) {
  constexpr int n = Rows<L, N>::kAll;
  return dim3((unsigned)((a.T + n - 1) / n), (unsigned)(a.c.batch * a.c.Hkv), 2);
}

template <int L, int N>
cudaError_t append(const CacheRowsArgs &a, cudaStream_t st) {
  const dim3 grid = row_grid<L, N>(a);
  switch (a.c.format) {
    case FS_CACHE_BF16: k11_append_kernel<FS_CACHE_BF16, L, N><<<grid, 256, 0, st>>>(a); break;
    case FS_CACHE_E4M3: k11_append_kernel<FS_CACHE_E4M3, L, N><<<grid, 256, 0, st>>>(a); break;
    case FS_CACHE_INT8: k11_append_kernel<FS_CACHE_INT8, L, N><<<grid, 256, 0, st>>>(a); break;
    default: k11_append_kernel<FS_CACHE_INT4, L, N><<<grid, 256, 0, st>>>(a); break;
  }
  return cudaGetLastError();
}

template <int L, int N, bool F32>
cudaError_t read(const CacheRowsArgs &a, cudaStream_t st) {
  const dim3 grid = row_grid<L, N>(a);
  switch (a.c.format) {
    case FS_CACHE_BF16: k11_read_kernel<FS_CACHE_BF16, L, N, F32><<<grid, 256, 0, st>>>(a); break;
    case FS_CACHE_E4M3: k11_read_kernel<FS_CACHE_E4M3, L, N, F32><<<grid, 256, 0, st>>>(a); break;
    case FS_CACHE_INT8: k11_read_kernel<FS_CACHE_INT8, L, N, F32><<<grid, 256, 0, st>>>(a); break;
    default: k11_read_kernel<FS_CACHE_INT4, L, N, F32><<<grid, 256, 0, st>>>(a); break;
  }
  return cudaGetLastError();
}

// Four rows a thread keep 128 bytes of loads in flight for the append (65536 x 16
// x 64 to e4m3 and back 140 us, two rows 146, one 163), two for the read (four:
// 143); with no more tokens than a block of single rows has, more would only idle
// threads.
template <int L>
bool few(const CacheRowsArgs &a) {
  return a.T <= Rows<L, 1>::kAll;
}

template <int L>
cudaError_t read_l(const CacheRowsArgs &a, cudaStream_t st) {
  if (few<L>(a)) return a.f32 ? read<L, 1, true>(a, st) : read<L, 1, false>(a, st);
  return a.f32 ? read<L, 2, true>(a, st) : read<L, 2, false>(a, st);
}

}  // namespace

cudaError_t launch_cache_append(const CacheRowsArgs &a, cudaStream_t st) {
  if (a.c.d == 64) return few<4>(a) ? append<4, 1>(a, st) : append<4, 4>(a, st);
  return few<8>(a) ? append<8, 1>(a, st) : append<8, 4>(a, st);
}

cudaError_t launch_cache_read(const CacheRowsArgs &a, cudaStream_t st) {
  return a.c.d == 64 ? read_l<4>(a, st) : read_l<8>(a, st);
}

cudaError_t launch_cache_accept(const CacheRowsArgs &a, cudaStream_t st) {
  const int words = (int)(fs_cache_row_bytes(a.c.d, a.c.format) / 16);
  const int threads = (a.T * words + 31) / 32 * 32;
  k11_accept_kernel<<<dim3(1, (unsigned)(a.c.batch * a.c.Hkv), 2), threads < 256 ? threads : 256, 0,
                      st>>>(a, words);
  return cudaGetLastError();
}

}  // namespace fs
