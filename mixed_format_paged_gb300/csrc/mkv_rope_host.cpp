// Host side of rotary positions: frequency tables and the checks of mkv_rope.
#include "mkv.h"
#include "mkv_internal.h"

#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstdlib>
#include <cstring>

namespace mkv {
int report(int status, const char* text);               // mkv_host.cpp
}

namespace {

using namespace mkv;

mkv_status fail(mkv_status st, const char* fmt, ...) {
  char buf[256];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  return mkv_status(report(st, buf));
}

// w / 2 pi modulo one turn, in units of 2^-64
uint64_t to_turns(double w) {
  const double t = w / (2.0 * M_PI);
  const double f = t - std::floor(t);                   // [0, 1]; 1 only for a tiny negative t
  const double hi = std::floor(f * 4294967296.0);
  const double lo = std::floor((f * 4294967296.0 - hi) * 4294967296.0 + 0.5);
  return (static_cast<uint64_t>(hi) << 32) + static_cast<uint64_t>(lo);
}

}  // namespace

extern "C" {

mkv_status mkv_rope_from_frequencies(int32_t rot_dim, int32_t interleaved, double mscale, const double* inv_freq,
                                     mkv_rope_table* table) {
  if (!table || !inv_freq) return fail(MKV_ERR_INVALID_ARGUMENT, "table or inv_freq is NULL");
  if (rot_dim < 2 || rot_dim > kMaxRot || rot_dim % 2)
    return fail(MKV_ERR_INVALID_ARGUMENT, "rot_dim %d outside 2..%d or odd", rot_dim, kMaxRot);
  if (!std::isfinite(mscale)) return fail(MKV_ERR_INVALID_ARGUMENT, "mscale is not finite");
  for (int i = 0; i < rot_dim / 2; ++i)
    if (!std::isfinite(inv_freq[i])) return fail(MKV_ERR_INVALID_ARGUMENT, "inv_freq[%d] is not finite", i);
  mkv_rope_table t;
  std::memset(&t, 0, sizeof t);
  t.rot_dim = rot_dim;
  t.interleaved = interleaved != 0;
  t.mscale = static_cast<float>(mscale);
  for (int i = 0; i < rot_dim / 2; ++i) {
    t.inv_freq[i] = inv_freq[i];
    t.turns[i] = to_turns(inv_freq[i]);
  }
  *table = t;
  return MKV_OK;
}

mkv_status mkv_rope_init(const mkv_rope_config* c, mkv_rope_table* table) {
  if (!c || !table) return fail(MKV_ERR_INVALID_ARGUMENT, "config or table is NULL");
  if (c->rot_dim < 2 || c->rot_dim > kMaxRot || c->rot_dim % 2)
    return fail(MKV_ERR_INVALID_ARGUMENT, "rot_dim %d outside 2..%d or odd", c->rot_dim, kMaxRot);
  if (c->reserved != 0) return fail(MKV_ERR_INVALID_ARGUMENT, "reserved field not 0");
  if (!std::isfinite(c->base) || !(c->base > 1.0)) return fail(MKV_ERR_INVALID_ARGUMENT, "base must be > 1");
  if (c->scaling < MKV_ROPE_NONE || c->scaling > MKV_ROPE_WAVELENGTH)
    return fail(MKV_ERR_INVALID_ARGUMENT, "scaling %d", c->scaling);
  if (c->scaling != MKV_ROPE_NONE && (!std::isfinite(c->factor) || !(c->factor >= 1.0)))
    return fail(MKV_ERR_INVALID_ARGUMENT, "factor must be >= 1");
  const bool ranged = c->scaling == MKV_ROPE_YARN || c->scaling == MKV_ROPE_WAVELENGTH;
  if (ranged && (!std::isfinite(c->original_length) || !(c->original_length >= 1.0)))
    return fail(MKV_ERR_INVALID_ARGUMENT, "original_length must be >= 1");
  if (c->scaling == MKV_ROPE_YARN &&
      (!std::isfinite(c->beta_fast) || !(c->beta_slow > 0.0) || !(c->beta_fast >= c->beta_slow)))
    return fail(MKV_ERR_INVALID_ARGUMENT, "beta_fast >= beta_slow > 0 is needed");
  if (c->scaling == MKV_ROPE_WAVELENGTH &&
      (!std::isfinite(c->high_freq) || !(c->low_freq > 0.0) || !(c->high_freq > c->low_freq)))
    return fail(MKV_ERR_INVALID_ARGUMENT, "high_freq > low_freq > 0 is needed");
  const int r = c->rot_dim, half = r / 2;
  double w[kMaxRot / 2], base = c->base, m = 1.0;
  if (c->scaling == MKV_ROPE_NTK) base *= std::pow(c->factor, double(r) / (r > 2 ? r - 2 : 1));
  for (int i = 0; i < half; ++i) w[i] = std::pow(base, -2.0 * i / r);
  if (c->scaling == MKV_ROPE_LINEAR)
    for (int i = 0; i < half; ++i) w[i] /= c->factor;
  if (c->scaling == MKV_ROPE_YARN) {
    // the pair index at which a pair makes `turns` turns over the original length
    auto at = [&](double turns) {
      return r * std::log(c->original_length / (turns * 2.0 * M_PI)) / (2.0 * std::log(c->base));
    };
    // (the ramp may end past the last pair, which then turns too fast to be slowed down by the whole factor)
    const double low = std::fmax(std::floor(at(c->beta_fast)), 0.0);
    const double high = std::fmin(std::ceil(at(c->beta_slow)), r - 1.0);
    for (int i = 0; i < half; ++i) {
      const double slow = std::fmin(std::fmax((i - low) / std::fmax(high - low, 1e-3), 0.0), 1.0);
      w[i] = w[i] / c->factor * slow + w[i] * (1.0 - slow);
    }
    m = 0.1 * std::log(c->factor) + 1.0;
  }
  if (c->scaling == MKV_ROPE_WAVELENGTH)
    for (int i = 0; i < half; ++i) {
      const double turns = c->original_length * w[i] / (2.0 * M_PI);
      const double keep = std::fmin(std::fmax((turns - c->low_freq) / (c->high_freq - c->low_freq), 0.0), 1.0);
      w[i] = w[i] * keep + w[i] / c->factor * (1.0 - keep);
    }
  return mkv_rope_from_frequencies(r, c->interleaved, m, w, table);
}

mkv_status mkv_rope(const mkv_rope_table* table, int64_t tokens, int32_t head_dim, const void* positions,
                    int32_t position_bytes, const mkv_rope_rows* q, const mkv_rope_rows* k, mkv_dtype dtype,
                    int32_t transpose, mkv_stream_t stream) {
  if (!table || !q) return fail(MKV_ERR_INVALID_ARGUMENT, "table or q is NULL");
  if (table->rot_dim < 2 || table->rot_dim > kMaxRot || table->rot_dim % 2)
    return fail(MKV_ERR_INVALID_ARGUMENT, "rot_dim %d outside 2..%d or odd", table->rot_dim, kMaxRot);
  if (dtype != MKV_F32 && dtype != MKV_BF16 && dtype != MKV_F16) return fail(MKV_ERR_INVALID_ARGUMENT, "dtype");
  if (position_bytes != 4 && position_bytes != 8) return fail(MKV_ERR_INVALID_ARGUMENT, "position_bytes %d", position_bytes);
  if (head_dim < table->rot_dim || head_dim > 4096)
    return fail(MKV_ERR_INVALID_ARGUMENT, "head_dim %d outside [rot_dim %d, 4096]", head_dim, table->rot_dim);
  if (tokens < 0 || tokens > (int64_t(1) << 40)) return fail(MKV_ERR_INVALID_ARGUMENT, "tokens");
  const size_t elt = dtype == MKV_F32 ? 4 : 2;
  RopeParams p;
  std::memset(&p, 0, sizeof p);
  for (int i = 0; i < 2; ++i) {
    const mkv_rope_rows* r = i ? k : q;
    const char* name = i ? "k" : "q";
    if (!r) continue;
    if (r->heads < 0 || r->heads > 4096 || r->reserved != 0) return fail(MKV_ERR_INVALID_ARGUMENT, "%s: heads %d", name, r->heads);
    if (tokens == 0 || r->heads == 0) continue;
    if (!r->in || !r->out) return fail(MKV_ERR_INVALID_ARGUMENT, "%s: in or out is NULL", name);
    if ((reinterpret_cast<uintptr_t>(r->in) | reinterpret_cast<uintptr_t>(r->out)) % elt)
      return fail(MKV_ERR_INVALID_ARGUMENT, "%s: address not aligned to its type", name);
    if (r->in_token < 0 || r->in_head < 0 || r->out_token < 0 || r->out_head < 0)
      return fail(MKV_ERR_INVALID_ARGUMENT, "%s: negative stride", name);
    // no two rows of the output overlap: heads inside a token, or tokens inside a head
    const __int128 over_heads = __int128(r->heads - 1) * r->out_head + head_dim;
    const __int128 over_tokens = __int128(tokens - 1) * r->out_token + head_dim;
    const bool heads_in = (r->heads == 1 || r->out_head >= head_dim) && (tokens == 1 || r->out_token >= over_heads);
    const bool tokens_in = (tokens == 1 || r->out_token >= head_dim) && (r->heads == 1 || r->out_head >= over_tokens);
    if (!heads_in && !tokens_in) return fail(MKV_ERR_INVALID_ARGUMENT, "%s: the output's rows overlap", name);
    if (r->in == r->out && ((tokens > 1 && r->in_token != r->out_token) || (r->heads > 1 && r->in_head != r->out_head)))
      return fail(MKV_ERR_INVALID_ARGUMENT, "%s: in place with other strides", name);
    (i ? p.k : p.q) = RopeRows{r->in, r->out, r->in_token, r->in_head, r->out_token, r->out_head, r->heads};
  }
  if (p.q.heads + p.k.heads == 0) return MKV_OK;
  if (!positions || reinterpret_cast<uintptr_t>(positions) % size_t(position_bytes))
    return fail(MKV_ERR_INVALID_ARGUMENT, "positions is NULL or not aligned");
  p.pos = positions;
  p.pos64 = position_bytes == 8;
  p.half = table->rot_dim / 2;
  p.inverse = transpose != 0;
  p.mscale = table->mscale;
  std::memcpy(p.turn, table->turns, size_t(p.half) * sizeof(uint64_t));
  const cudaError_t e = launch_rope(p, tokens, head_dim, dtype, table->interleaved != 0, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(MKV_ERR_CUDA, "rope launch: %s", cudaGetErrorString(e));
  return MKV_OK;
}

}  // extern "C"
