// cache_api.cpp -- the C ABI of the page-cache operators (pkd_append, pkd_gather, pkd_copy_pages)
// and the bookkeeping of a pool's pages (pkd_pages_*).
#include <cuda_runtime.h>

#include <cfloat>
#include <cstdint>
#include <cstring>
#include <exception>
#include <new>
#include <string>
#include <utility>
#include <vector>

#include "cache_ops.cuh"

namespace pkd {
void set_error_message(const char* msg);
}

using namespace pkd;

namespace {

int bad(const std::string& msg, int code = PKD_ERR_INVALID_ARG) {
  set_error_message(msg.c_str());
  return code;
}

int done(cudaError_t e, const char* what) {
  if (e == cudaSuccess) {
    set_error_message("");
    return PKD_OK;
  }
  return bad(std::string(what) + ": " + cudaGetErrorString(e), PKD_ERR_CUDA);
}

bool on16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// A failing call must not throw across the C boundary (the messages allocate).
template <typename F>
int guarded(F f) {
  try {
    return f();
  } catch (const std::bad_alloc&) {
    set_error_message("out of host memory");
    return PKD_ERR_INVALID_ARG;
  } catch (const std::exception& e) {
    set_error_message(e.what());
    return PKD_ERR_INVALID_ARG;
  }
}

int check_pool(const pkd_paged_pool& p, int io_dtype, bool used) {
  if (io_dtype != PKD_DTYPE_F16 && io_dtype != PKD_DTYPE_BF16)
    return bad("rows outside the cache are F16 or BF16");
  if (p.head_dim != 64 && p.head_dim != 128 && p.head_dim != 256)
    return bad("head_dim must be 64, 128 or 256", PKD_ERR_UNSUPPORTED);
  if (!used) return PKD_OK;
  if (p.dtype != io_dtype && p.dtype != PKD_DTYPE_E4M3 && p.dtype != PKD_DTYPE_E2M1)
    return bad("the cache's dtype must be that of the rows, E4M3 or E2M1", PKD_ERR_UNSUPPORTED);
  if (p.page_size < 8 || p.page_size > 256 || (p.page_size & (p.page_size - 1)) != 0)
    return bad("page_size must be a power of two in [8, 256]", PKD_ERR_UNSUPPORTED);
  if (p.num_kv_heads <= 0 || p.num_kv_heads > (1 << 20)) return bad("num_kv_heads must be positive");
  if (p.num_pages <= 0 || p.num_pages > (int64_t(1) << 31))
    return bad("num_pages must lie in [1, 2^31]");
  if (p.batch < 0 || p.num_indices < 0 || !p.indptr || (p.num_indices > 0 && !p.indices))
    return bad("the page table is malformed or null");
  if (!p.k || !p.v) return bad("null k / v pool");
  if (!on16(p.k) || !on16(p.v)) return bad("the K/V pools must be 16-byte aligned");
  const int elt = p.dtype == PKD_DTYPE_F16 || p.dtype == PKD_DTYPE_BF16 ? 2 : 1;
  for (int i = 0; i < 3; ++i)
    if (p.strides[i] <= 0 || p.strides[i] * elt % 16 != 0)
      return bad("kv strides must be positive multiples of 16 bytes");
  if (p.dtype == PKD_DTYPE_E2M1) {
    const int sb = p.head_dim / 16;
    if (!p.k_scales || !p.v_scales) return bad("an E2M1 cache needs its scale pools");
    if (reinterpret_cast<uintptr_t>(p.k_scales) % sb || reinterpret_cast<uintptr_t>(p.v_scales) % sb)
      return bad("the scale pools must be aligned to head_dim / 16 bytes");
    for (int i = 0; i < 3; ++i)
      if (p.scale_strides[i] <= 0 || p.scale_strides[i] % sb != 0)
        return bad("scale strides must be positive multiples of head_dim / 16 bytes");
  }
  for (float s : {p.k_scale, p.v_scale})
    if (!(s >= 5.4210109e-20f && s <= 1.8446744e19f))  // 2^-64 .. 2^64: no quotient over- or underflows
      return bad("k_scale and v_scale must lie in [2^-64, 2^64]");
  return PKD_OK;
}

// Whether rows of `row` units at these strides of (page, slot, head) lie apart: each axis clears what the
// shorter ones span.
bool rows_apart(const pkd_paged_pool& p, const int64_t (&st)[3], int64_t row) {
  int64_t axis[3][2] = {{st[0], p.num_pages}, {st[1], p.page_size}, {st[2], p.num_kv_heads}};
  for (int i = 0; i < 2; ++i)
    for (int j = 0; j < 2 - i; ++j)
      if (axis[j][0] > axis[j + 1][0]) std::swap(axis[j], axis[j + 1]);
  for (auto& a : axis) {
    if (a[1] <= 1) continue;
    if (a[0] < row) return false;
    row += (a[1] - 1) * a[0];
  }
  return true;
}

// A pool that is written: no two of its rows may share bytes.
int check_written(const pkd_paged_pool& p) {
  const bool codes = p.dtype == PKD_DTYPE_E2M1;
  if (p.k == p.v || !rows_apart(p, p.strides, codes ? p.head_dim / 2 : p.head_dim))
    return bad("the K and V pools are one, or their rows overlap");
  if (codes && (p.k_scales == p.v_scales || !rows_apart(p, p.scale_strides, p.head_dim / 16)))
    return bad("the scale pools are one, or their rows overlap");
  return PKD_OK;
}

int check_rows(const void* p, const int64_t (&st)[2], const char* name) {
  if (!p) return bad(std::string(name) + " is null");
  if (!on16(p)) return bad(std::string(name) + " must be 16-byte aligned");
  if (st[0] < 0 || st[1] < 0 || st[0] % 8 != 0 || st[1] % 8 != 0)
    return bad(std::string(name) + " strides must be multiples of 8 elements");
  return PKD_OK;
}

// Rows that are written: no two may share bytes.
int check_out(const void* p, const int64_t (&st)[2], int64_t tokens, int64_t heads, int head_dim,
              const char* name) {
  if (int rc = check_rows(p, st, name)) return rc;
  const int64_t D = head_dim;
  const bool by_token = (heads <= 1 || st[1] >= D) && (tokens <= 1 || st[0] >= (heads - 1) * st[1] + D);
  const bool by_head = (tokens <= 1 || st[0] >= D) && (heads <= 1 || st[1] / (tokens > 1 ? tokens - 1 : 1) >= st[0] &&
                                                        st[1] - (tokens - 1) * st[0] >= D);
  if (!by_token && !by_head) return bad(std::string(name) + ": its rows overlap");
  return PKD_OK;
}

// Whether a row of a and a row of b (n tokens of ha and hb heads, checked strides) share bytes; where
// their tokens lie at different distances (or it would take long to tell), whether the memory that they
// span does.
bool rows_overlap(const void* a, const int64_t (&sa)[2], int64_t ha, const void* b, const int64_t (&sb)[2],
                  int64_t hb, int64_t n, int64_t D) {
  if (ha == 0 || hb == 0) return false;
  const int64_t a0 = n > 1 ? sa[0] : 0, b0 = n > 1 ? sb[0] : 0, a1 = ha > 1 ? sa[1] : 0, b1 = hb > 1 ? sb[1] : 0;
  const int64_t off = (static_cast<const char*>(b) - static_cast<const char*>(a)) / 2;
  if (off >= (n - 1) * a0 + (ha - 1) * a1 + D || -off >= (n - 1) * b0 + (hb - 1) * b1 + D) return false;
  const bool even = a1 == b1 || ha == 1 || hb == 1;
  if (a0 != b0 || (!even && ha * hb > 65536)) return true;
  // two rows start off + jb * b1 - ja * a1 + i * a0 elements apart, |i| < n
  auto meet = [&](int64_t x) {
    const int64_t i = a0 > 0 ? (x < 0 ? -((a0 - 1 - x) / a0) : x / a0) : 0;  // x - i * a0 in [0, a0)
    return (i < n && -i < n && x - i * a0 < D && x - i * a0 > -D) ||
           (a0 > 0 && i + 1 < n && -(i + 1) < n && (i + 1) * a0 - x < D);
  };
  if (even) {
    const int64_t st = ha == 1 ? b1 : a1;
    for (int64_t j = 1 - ha; j < hb; ++j)
      if (meet(off + j * st)) return true;
    return false;
  }
  for (int64_t ja = 0; ja < ha; ++ja)
    for (int64_t jb = 0; jb < hb; ++jb)
      if (meet(off + jb * b1 - ja * a1)) return true;
  return false;
}

bool same_rows(const void* a, const int64_t (&sa)[2], const void* b, const int64_t (&sb)[2], int64_t n, int64_t heads) {
  return a == b && (n <= 1 || sa[0] == sb[0]) && (heads <= 1 || sa[1] == sb[1]);
}

}  // namespace

extern "C" int pkd_append(const pkd_append_args* args, void* stream) {
  return guarded([&]() -> int {
    if (!args) return bad("args is null");
    const pkd_append_args& a = *args;
    const bool kv = a.k != nullptr || a.v != nullptr;
    if (int rc = check_pool(a.pool, a.in_dtype, kv)) return rc;
    if (a.num_tokens < 0) return bad("num_tokens must be >= 0");
    if (a.num_qo_heads < 0 || a.num_qo_heads > (1 << 20)) return bad("num_qo_heads must be >= 0");
    if (a.num_tokens == 0) return done(cudaSuccess, "");  // (tensors of no rows have no address)
    if ((a.q != nullptr) != (a.num_qo_heads > 0)) return bad("q and num_qo_heads do not agree");
    if ((a.k != nullptr) != (a.v != nullptr)) return bad("k and v come together");
    if (!kv && a.pool.num_kv_heads != 0) return bad("num_kv_heads without k and v");
    if (!kv && !a.q) return bad("neither q nor k and v are given");
    if (a.q) {
      if (int rc = check_rows(a.q, a.q_strides, "q")) return rc;
      if (int rc = check_out(a.q_out, a.q_out_strides, a.num_tokens, a.num_qo_heads, a.pool.head_dim, "q_out")) return rc;
    }
    if (kv) {
      if (int rc = check_written(a.pool)) return rc;
      if (int rc = check_rows(a.k, a.k_strides, "k")) return rc;
      if (int rc = check_rows(a.v, a.v_strides, "v")) return rc;
    }
    if (a.q) {
      const int64_t n = a.num_tokens, hq = a.num_qo_heads, hkv = a.pool.num_kv_heads, D = a.pool.head_dim;
      if ((!same_rows(a.q_out, a.q_out_strides, a.q, a.q_strides, n, hq) &&
           rows_overlap(a.q_out, a.q_out_strides, hq, a.q, a.q_strides, hq, n, D)) ||
          (kv && (rows_overlap(a.q_out, a.q_out_strides, hq, a.k, a.k_strides, hkv, n, D) ||
                  rows_overlap(a.q_out, a.q_out_strides, hq, a.v, a.v_strides, hkv, n, D))))
        return bad("q_out overlaps rows of q (other than being q), k or v");
    }
    if (!a.batch_indices || !a.positions) return bad("null batch_indices / positions");
    if ((a.q_weight && !on16(a.q_weight)) || (a.k_weight && !on16(a.k_weight)))
      return bad("the norm weights must be 16-byte aligned");
    if (!(a.eps == 0.0 || (a.eps >= FLT_MIN && a.eps <= FLT_MAX)))
      return bad("eps must be 0 or a normal 32-bit number");
    if (a.rotary_dim < 0 || a.rotary_dim > a.pool.head_dim || a.rotary_dim % 16 != 0)
      return bad("rotary_dim must be 0 or a multiple of 16 up to head_dim");
    if (a.rotary_dim > 0 && (!a.cos_sin || !on16(a.cos_sin) || a.cos_sin_rows < 0))
      return bad("cos_sin must be a 16-byte aligned table when rotary_dim > 0");
    return done(launch_append(a, static_cast<cudaStream_t>(stream)), "append kernel launch");
  });
}

extern "C" int pkd_gather(const pkd_gather_args* args, void* stream) {
  return guarded([&]() -> int {
    if (!args) return bad("args is null");
    const pkd_gather_args& a = *args;
    if (int rc = check_pool(a.pool, a.out_dtype, true)) return rc;
    if (a.num_tokens < 0) return bad("num_tokens must be >= 0");
    if (a.num_tokens == 0) return done(cudaSuccess, "");
    if (!a.k_out && !a.v_out) return bad("k_out and v_out are both null");
    if (a.k_out)
      if (int rc = check_out(a.k_out, a.k_out_strides, a.num_tokens, a.pool.num_kv_heads, a.pool.head_dim, "k_out"))
        return rc;
    if (a.v_out)
      if (int rc = check_out(a.v_out, a.v_out_strides, a.num_tokens, a.pool.num_kv_heads, a.pool.head_dim, "v_out"))
        return rc;
    if (a.k_out && a.v_out &&
        rows_overlap(a.k_out, a.k_out_strides, a.pool.num_kv_heads, a.v_out, a.v_out_strides, a.pool.num_kv_heads,
                     a.num_tokens, a.pool.head_dim))
      return bad("k_out overlaps v_out");
    if (!a.batch_indices || !a.positions) return bad("null batch_indices / positions");
    return done(launch_gather(a, static_cast<cudaStream_t>(stream)), "gather kernel launch");
  });
}

extern "C" int pkd_evict(const pkd_evict_args* args, void* stream) {
  return guarded([&]() -> int {
    if (!args) return bad("args is null");
    const pkd_evict_args& a = *args;
    const int dt = a.pool.dtype;
    if (int rc = check_pool(a.pool, dt == PKD_DTYPE_BF16 ? PKD_DTYPE_BF16 : PKD_DTYPE_F16, true)) return rc;
    if (int rc = check_written(a.pool)) return rc;
    if (a.budget < 1 || a.budget > 1 << 30) return bad("budget must lie in [1, 2^30]");
    if (a.num_sink_tokens < 0 || a.num_recent < 0 || (int64_t)a.num_sink_tokens + a.num_recent > a.budget)
      return bad("num_sink_tokens and num_recent must be >= 0 and fit the budget together");
    if (a.pool.batch == 0) return done(cudaSuccess, "");
    if ((int64_t)a.pool.batch * a.pool.num_kv_heads > INT32_MAX) return bad("batch * num_kv_heads is too large");
    if (!a.kv_lens) return bad("null kv_lens");
    if (!a.key_weights || reinterpret_cast<uintptr_t>(a.key_weights) % 4) return bad("key_weights is null or not aligned");
    const int64_t n[3] = {a.pool.num_pages, a.pool.num_kv_heads, a.pool.page_size};
    for (int i = 0; i < 3; ++i)
      if (a.weight_strides[i] < 0 || (n[i] > 1 && a.weight_strides[i] > (int64_t(1) << 60) / n[i]))
        return bad("key_weights strides must be positive, within 2^60 elements");
    const int64_t st[3] = {a.weight_strides[0], a.weight_strides[2], a.weight_strides[1]};
    if (!rows_apart(a.pool, st, 1)) return bad("entries of key_weights overlap");
    // (page and slot strides are held in 32 bits: of 16 bytes, of 4 for scales, of an element for weights)
    const int64_t unit = dt == PKD_DTYPE_F16 || dt == PKD_DTYPE_BF16 ? 8 : 16;
    for (int i = 0; i < 2; ++i) {
      const int64_t entries = i == 0 ? a.pool.num_pages : a.pool.page_size;
      if (entries > 1 && (a.pool.strides[i] / unit > UINT32_MAX || st[i] > UINT32_MAX ||
                          (dt == PKD_DTYPE_E2M1 && a.pool.scale_strides[i] / 4 > UINT32_MAX)))
        return bad("page or slot strides of more than 2^32 units");
    }
    if (!a.moves && a.num_sink_tokens + a.num_recent < a.budget) return bad("moves is null");
    if (reinterpret_cast<uintptr_t>(a.moves) % 8) return bad("moves must be 8-byte aligned");
    return done(launch_evict(a, static_cast<cudaStream_t>(stream)), "evict kernel launch");
  });
}

extern "C" int pkd_copy_pages(void* const* bases, const int64_t* page_strides,
                              const int64_t* page_bytes, int n_pools, int64_t num_pages,
                              const int32_t* src_pages, const int32_t* dst_pages, int64_t n_pairs,
                              void* stream) {
  return guarded([&]() -> int {
    if (n_pools < 0 || n_pairs < 0 || num_pages < 0 || num_pages > (int64_t(1) << 31))
      return bad("negative count, or more than 2^31 pages");
    if (n_pools > 0 && (!bases || !page_strides || !page_bytes)) return bad("null pool table");
    if (n_pairs > 0 && (!src_pages || !dst_pages)) return bad("null src_pages / dst_pages");
    // A page is a source or a destination, and a destination once.  The ids lie in a table of bits
    // of the pool's size.
    std::vector<uint64_t> is_dst((size_t)(num_pages + 63) / 64);
    for (int64_t i = 0; i < n_pairs; ++i) {
      const int64_t s = src_pages[i], d = dst_pages[i];
      if (s < 0 || s >= num_pages || d < 0 || d >= num_pages)
        return bad("pair " + std::to_string(i) + ": page id outside [0, " + std::to_string(num_pages) + ")");
      uint64_t& w = is_dst[(size_t)(d >> 6)];
      if (w >> (d & 63) & 1)
        return bad("pair " + std::to_string(i) + ": page " + std::to_string(d) + " is a destination twice");
      w |= uint64_t(1) << (d & 63);
    }
    for (int64_t i = 0; i < n_pairs; ++i)
      if (is_dst[(size_t)(src_pages[i] >> 6)] >> (src_pages[i] & 63) & 1)
        return bad("pair " + std::to_string(i) + ": page " + std::to_string(src_pages[i]) +
                   " is a source and a destination");
    std::vector<CopyPool> pools;
    for (int j = 0; j < n_pools; ++j) {
      if (page_bytes[j] < 0 || page_strides[j] < page_bytes[j])
        return bad("pool " + std::to_string(j) + ": page_stride must be >= page_bytes >= 0");
      if (page_bytes[j] > (int64_t(1) << 36))
        return bad("pool " + std::to_string(j) + ": pages of more than 64 GiB");
      if (page_bytes[j] == 0) continue;
      if (!bases[j]) return bad("pool " + std::to_string(j) + " is null");
      pools.push_back({static_cast<char*>(bases[j]), page_strides[j], page_bytes[j]});
    }
    if (n_pairs == 0 || pools.empty()) return done(cudaSuccess, "");
    return done(launch_copy_pages(pools.data(), (int)pools.size(), src_pages, dst_pages, n_pairs,
                                  static_cast<cudaStream_t>(stream)),
                "page copy launch");
  });
}

// ------------------------------------------------------------------------------ page bookkeeping
// uses[p]: sequences that own page p; free pages also have their bit set, and no word below
// `hint` holds a free page, so that the lowest free page is found without a search from 0.
struct pkd_pages {
  std::vector<int32_t> uses;
  std::vector<uint64_t> free_bits;
  int64_t n_free = 0;
  size_t hint = 0;

  int32_t take() {  // n_free > 0
    while (free_bits[hint] == 0) ++hint;
    const int bit = __builtin_ctzll(free_bits[hint]);
    free_bits[hint] &= free_bits[hint] - 1;
    --n_free;
    const int32_t page = (int32_t)(hint * 64 + bit);
    uses[(size_t)page] = 1;
    return page;
  }
  void drop(int32_t page) {  // uses[page] > 0
    if (--uses[(size_t)page] > 0) return;
    const size_t w = (size_t)page / 64;
    free_bits[w] |= uint64_t(1) << (page % 64);
    ++n_free;
    if (w < hint) hint = w;
  }
  bool known(int32_t page) const { return page >= 0 && (size_t)page < uses.size(); }
};

extern "C" int pkd_pages_create(pkd_pages** out, int64_t num_pages) {
  return guarded([&]() -> int {
    if (!out) return bad("out is null");
    *out = nullptr;
    if (num_pages < 0 || num_pages > INT32_MAX) return bad("num_pages must lie in [0, 2^31)");
    pkd_pages* p = new pkd_pages();
    try {
      p->uses.assign((size_t)num_pages, 0);
      p->free_bits.assign((size_t)(num_pages + 63) / 64, ~uint64_t(0));
    } catch (...) {
      delete p;
      throw;
    }
    if (num_pages % 64) p->free_bits.back() = (uint64_t(1) << (num_pages % 64)) - 1;
    p->n_free = num_pages;
    *out = p;
    set_error_message("");
    return PKD_OK;
  });
}

extern "C" int pkd_pages_destroy(pkd_pages* p) {
  delete p;
  return PKD_OK;
}

extern "C" int pkd_pages_alloc(pkd_pages* p, int64_t n, int32_t* out) {
  return guarded([&]() -> int {
    if (!p || n < 0 || (n > 0 && !out)) return bad("null pages / out, or n < 0");
    if (n > p->n_free)
      return bad("asked for " + std::to_string(n) + " pages, " + std::to_string(p->n_free) + " are free");
    for (int64_t i = 0; i < n; ++i) out[i] = p->take();
    return PKD_OK;
  });
}

extern "C" int pkd_pages_free(pkd_pages* p, const int32_t* pages, int64_t n) {
  return guarded([&]() -> int {
    if (!p || n < 0 || (n > 0 && !pages)) return bad("null pages, or n < 0");
    for (int64_t i = 0; i < n; ++i) {
      if (!p->known(pages[i]) || p->uses[(size_t)pages[i]] == 0) {
        for (int64_t j = 0; j < i; ++j) ++p->uses[(size_t)pages[j]];  // take the counts back
        return bad("pages[" + std::to_string(i) + "] = " + std::to_string(pages[i]) +
                   " is not in use (so often)");
      }
      --p->uses[(size_t)pages[i]];
    }
    for (int64_t i = 0; i < n; ++i) ++p->uses[(size_t)pages[i]];
    for (int64_t i = 0; i < n; ++i) p->drop(pages[i]);
    return PKD_OK;
  });
}

extern "C" int pkd_pages_fork(pkd_pages* p, const int32_t* pages, int64_t n_pages, int64_t kv_len,
                              int page_size, int32_t* out, int32_t* copy_src, int32_t* copy_dst) {
  return guarded([&]() -> int {
    if (!p || !copy_src || !copy_dst || n_pages < 0 || (n_pages > 0 && !pages))
      return bad("null argument, or n_pages < 0");
    if (page_size < 1 || kv_len < 0) return bad("page_size must be >= 1 and kv_len >= 0");
    const int64_t need = kv_len / page_size + (kv_len % page_size != 0);
    if (need > n_pages) return bad("kv_len tokens need more pages than the sequence owns");
    if (need > 0 && !out) return bad("out is null");
    for (int64_t i = 0; i < need; ++i) {
      if (!p->known(pages[i]) || p->uses[(size_t)pages[i]] == 0)
        return bad("pages[" + std::to_string(i) + "] = " + std::to_string(pages[i]) + " is not in use");
      if (p->uses[(size_t)pages[i]] == INT32_MAX) return bad("a page has 2^31 - 1 uses already");
    }
    *copy_src = *copy_dst = -1;
    const bool partial = kv_len % page_size != 0;
    if (partial && p->n_free == 0) return bad("no page is free for the partly filled last one");
    const int64_t shared = need - (partial ? 1 : 0);
    for (int64_t i = 0; i < shared; ++i) {
      ++p->uses[(size_t)pages[i]];
      out[i] = pages[i];
    }
    if (partial) {
      *copy_src = pages[shared];
      out[shared] = *copy_dst = p->take();
    }
    return PKD_OK;
  });
}

extern "C" int pkd_pages_compact(pkd_pages* p, int32_t* src, int32_t* dst, int64_t* n_moves,
                                 int32_t* remap) {
  return guarded([&]() -> int {
    if (!p || !n_moves) return bad("null argument");
    const int64_t total = (int64_t)p->uses.size();
    if (total > 0 && (!src || !dst || !remap)) return bad("null src / dst / remap");
    for (int64_t i = 0; i < total; ++i) remap[i] = (int32_t)i;
    const int64_t live = total - p->n_free;
    int64_t lo = 0, hi = total - 1, n = 0;
    while (true) {  // the highest page in use goes to the lowest free one
      while (lo < live && p->uses[(size_t)lo] != 0) ++lo;
      while (hi >= live && p->uses[(size_t)hi] == 0) --hi;
      if (lo >= live) break;
      src[n] = (int32_t)hi;
      dst[n] = (int32_t)lo;
      ++n;
      remap[hi] = (int32_t)lo;
      p->uses[(size_t)lo] = p->uses[(size_t)hi];
      p->uses[(size_t)hi] = 0;
    }
    for (size_t w = 0; w < p->free_bits.size(); ++w) p->free_bits[w] = 0;
    for (int64_t i = live; i < total; ++i) p->free_bits[(size_t)i / 64] |= uint64_t(1) << (i % 64);
    p->hint = (size_t)live / 64;
    *n_moves = n;
    return PKD_OK;
  });
}

extern "C" int pkd_pages_count(pkd_pages* p, int64_t* n_free, int32_t* uses) {
  return guarded([&]() -> int {
    if (!p) return bad("pages is null");
    if (n_free) *n_free = p->n_free;
    if (uses && !p->uses.empty()) std::memcpy(uses, p->uses.data(), p->uses.size() * sizeof(int32_t));
    return PKD_OK;
  });
}
