// C ABI of the rotary positions and of the cache append that rotates on the way.
#include <cmath>
#include <cstdint>
#include <new>

#include "../../include/pa.h"
#include "pa_internal.h"

using namespace pa;

struct pa_rope_s {
    RopeParams params{};
    double freq[kMaxRotaryDim / 2] = {};   // angle per position of each pair
    double mag = 1.0;
};

namespace {

constexpr double kTwoPi = 6.283185307179586476925286766559;
constexpr double kTwoPiLow = 2.4492935982947064e-16;   // 2 pi - kTwoPi

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
bool positive(double x) { return x > 0 && std::isfinite(x); }

// rows [T][heads][D] with a token stride in elements, read and written in
// 16-byte pieces
bool good_rows(const void *p, int64_t stride, int64_t heads, int64_t d) {
    return p != nullptr && aligned(p, 16) && stride >= heads * d && stride % 8 == 0;
}

pa_status make_frequencies(const pa_rope_desc *d, pa_rope_s *r) {
    const int n = d->rotary_dim / 2;
    for (int i = 0; i < n; ++i) r->freq[i] = std::pow(d->base, -2.0 * i / d->rotary_dim);
    r->mag = 1.0;
    switch (d->scaling) {
        case PA_ROPE_SCALE_NONE: break;
        case PA_ROPE_SCALE_LINEAR:
            for (int i = 0; i < n; ++i) r->freq[i] /= d->factor;
            break;
        case PA_ROPE_SCALE_WAVELENGTH:
            for (int i = 0; i < n; ++i) {
                const double turns = d->original_max_position * r->freq[i] / kTwoPi;
                const double m = std::fmin(1.0, std::fmax(0.0, (turns - d->low) / (d->high - d->low)));
                r->freq[i] = r->freq[i] / d->factor * (1 - m) + r->freq[i] * m;
            }
            break;
        case PA_ROPE_SCALE_YARN: {
            // the (fractional) pair that makes `turns` turns over the original context
            auto at = [&](double turns) {
                return d->rotary_dim * std::log(d->original_max_position / (turns * kTwoPi)) / (2 * std::log(d->base));
            };
            const double lo = std::fmax(0.0, std::floor(at(d->high)));
            const double hi = std::fmin(d->rotary_dim - 1.0, std::ceil(at(d->low)));
            for (int i = 0; i < n; ++i) {
                const double ramp = std::fmin(1.0, std::fmax(0.0, (i - lo) / std::fmax(hi - lo, 1e-3)));
                r->freq[i] = r->freq[i] / d->factor * ramp + r->freq[i] * (1 - ramp);
            }
            r->mag = 0.1 * std::log(d->factor) + 1.0;
            break;
        }
    }
    if (d->attention_factor > 0) r->mag = d->attention_factor;
    for (int i = 0; i < n; ++i) {
        if (!std::isfinite(r->freq[i]) || r->freq[i] < 0) return PA_ERR_INVALID_ARGUMENT;
        // the fraction of a turn per position, as 64-bit fixed point (a whole
        // turn more or less changes nothing): the quotient, and what its
        // rounding left over, so that 2^31 positions stay below 2^-32 of a turn
        const double turns = r->freq[i] / kTwoPi;
        const double rest = (std::fma(-turns, kTwoPi, r->freq[i]) - turns * kTwoPiLow) / kTwoPi;
        const double frac = turns - std::floor(turns);
        if (!(turns < 0x1p40)) return PA_ERR_INVALID_ARGUMENT;   // too little of the fraction is left
        r->params.step[i] = static_cast<uint64_t>(std::ldexp(frac, 64)) +
                            static_cast<uint64_t>(static_cast<int64_t>(std::ldexp(rest, 64)));
    }
    r->params.mag = static_cast<float>(r->mag);
    if (!std::isfinite(r->params.mag)) return PA_ERR_INVALID_ARGUMENT;
    r->params.rotary_dim = d->rotary_dim;
    r->params.interleaved = d->layout == PA_ROPE_INTERLEAVED ? 1 : 0;
    return PA_OK;
}

}  // namespace

extern "C" {

pa_status pa_rope_create(const pa_rope_desc *d, pa_rope_t **out) {
    if (out) *out = nullptr;
    if (d == nullptr || out == nullptr) return PA_ERR_INVALID_ARGUMENT;
    if (d->rotary_dim <= 0 || d->rotary_dim % 2 != 0 || !positive(d->base)) return PA_ERR_INVALID_ARGUMENT;
    if (d->layout != PA_ROPE_HALF && d->layout != PA_ROPE_INTERLEAVED) return PA_ERR_INVALID_ARGUMENT;
    if (d->scaling < PA_ROPE_SCALE_NONE || d->scaling > PA_ROPE_SCALE_YARN) return PA_ERR_INVALID_ARGUMENT;
    if (!(d->attention_factor >= 0) || !std::isfinite(d->attention_factor)) return PA_ERR_INVALID_ARGUMENT;
    if (d->scaling != PA_ROPE_SCALE_NONE && !positive(d->factor)) return PA_ERR_INVALID_ARGUMENT;
    if (d->scaling == PA_ROPE_SCALE_WAVELENGTH || d->scaling == PA_ROPE_SCALE_YARN)
        if (!positive(d->low) || !positive(d->high) || !(d->low < d->high) || !(d->original_max_position > 0))
            return PA_ERR_INVALID_ARGUMENT;
    if (d->scaling == PA_ROPE_SCALE_YARN && !(d->base > 1)) return PA_ERR_INVALID_ARGUMENT;
    if (d->rotary_dim % 8 != 0 || d->rotary_dim > kMaxRotaryDim) return PA_ERR_UNSUPPORTED;
    pa_rope_s *r = new (std::nothrow) pa_rope_s();
    if (!r) return PA_ERR_INVALID_ARGUMENT;
    const pa_status st = make_frequencies(d, r);
    if (st != PA_OK) {
        delete r;
        return st;
    }
    *out = r;
    return PA_OK;
}

void pa_rope_destroy(pa_rope_t *rope) { delete rope; }

pa_status pa_rope_frequencies(const pa_rope_t *rope, double *frequencies, double *magnitude) {
    if (!rope || (!frequencies && !magnitude)) return PA_ERR_INVALID_ARGUMENT;
    if (frequencies)
        for (int i = 0; i < rope->params.rotary_dim / 2; ++i) frequencies[i] = rope->freq[i];
    if (magnitude) *magnitude = rope->mag;
    return PA_OK;
}

pa_status pa_rotary(const pa_rope_t *rope, const void *x, int64_t x_stride, const int32_t *positions, int32_t num_tokens,
                    int32_t num_heads, int32_t head_dim, void *out, int64_t out_stride, void *stream) {
    if (!rope || num_tokens < 0 || num_heads <= 0 || head_dim <= 0) return PA_ERR_INVALID_ARGUMENT;
    if (rope->params.rotary_dim > head_dim) return PA_ERR_INVALID_ARGUMENT;
    if (head_dim % 8 != 0 || head_dim > kMaxRotaryDim || num_heads > 65536) return PA_ERR_UNSUPPORTED;
    if (num_tokens == 0) return PA_OK;
    if (!good_rows(x, x_stride, num_heads, head_dim) || !good_rows(out, out_stride, num_heads, head_dim) || !positions ||
        !aligned(positions, 4))
        return PA_ERR_INVALID_ARGUMENT;
    RotaryParams p{};
    p.x = static_cast<const uint16_t *>(x);
    p.out = static_cast<uint16_t *>(out);
    p.positions = positions;
    p.x_stride = x_stride;
    p.out_stride = out_stride;
    p.num_tokens = num_tokens;
    p.num_heads = num_heads;
    p.head_dim = head_dim;
    return launch_rotary(rope->params, p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

pa_status pa_append_kv(const pa_rope_t *rope, const pa_append_args *a, void *stream) {
    if (!a) return PA_ERR_INVALID_ARGUMENT;
    if (a->num_reqs < 0 || a->num_tokens < 0 || a->num_heads_q < 0 || a->num_heads_kv <= 0 || a->head_dim <= 0 ||
        a->num_blocks <= 0 || a->max_blocks_per_req <= 0 || a->block_size <= 0)
        return PA_ERR_INVALID_ARGUMENT;
    int kind = -1;
    switch (a->kv_cache_dtype) {
        case PA_KV_BF16: kind = kCacheBf16; break;
        case PA_KV_FP8_E4M3: kind = kCacheE4m3; break;
        case PA_KV_FP8_E4M3_BLOCK: kind = kCacheE4m3Block; break;
        case PA_KV_INT8_BLOCK: kind = kCacheInt8Block; break;
        default: return PA_ERR_INVALID_ARGUMENT;
    }
    if (kind == kCacheE4m3 && (!positive(a->k_scale) || !positive(a->v_scale))) return PA_ERR_INVALID_ARGUMENT;
    if (rope && rope->params.rotary_dim > a->head_dim) return PA_ERR_INVALID_ARGUMENT;
    if (a->q && (!rope || a->num_heads_q <= 0)) return PA_ERR_INVALID_ARGUMENT;   // q is here to be rotated
    if (a->block_size != kBlockSize || (a->head_dim != 64 && a->head_dim != 128)) return PA_ERR_UNSUPPORTED;
    if (static_cast<int64_t>(a->num_blocks) * kBlockSize > INT32_MAX || a->num_heads_kv > 65536 || a->num_heads_q > 65536 ||
        a->num_reqs > INT32_MAX / 4)
        return PA_ERR_UNSUPPORTED;
    if (a->num_tokens == 0) return PA_OK;
    const int64_t hkv = a->num_heads_kv, hq = a->num_heads_q, d = a->head_dim;
    if (a->num_reqs == 0 || !a->query_start_loc || !a->num_computed_tokens || !a->block_table ||
        !aligned(a->query_start_loc, 4) || !aligned(a->num_computed_tokens, 4) || !aligned(a->block_table, 4))
        return PA_ERR_INVALID_ARGUMENT;
    if (!good_rows(a->key, a->key_stride, hkv, d) || !good_rows(a->value, a->value_stride, hkv, d))
        return PA_ERR_INVALID_ARGUMENT;
    if (!a->key_cache || !a->value_cache || !aligned(a->key_cache, 16) || !aligned(a->value_cache, 16))
        return PA_ERR_INVALID_ARGUMENT;
    if (a->q && (!good_rows(a->q, a->q_stride, hq, d) || !good_rows(a->q_out, a->q_out_stride, hq, d)))
        return PA_ERR_INVALID_ARGUMENT;
    const bool block_scaled = kind == kCacheE4m3Block || kind == kCacheInt8Block;
    if (block_scaled && (!a->key_scales || !a->value_scales || !aligned(a->key_scales, 4) || !aligned(a->value_scales, 4)))
        return PA_ERR_INVALID_ARGUMENT;
    AppendParams p{};
    p.q = static_cast<const uint16_t *>(a->q);
    p.q_out = static_cast<uint16_t *>(a->q_out);
    p.key = static_cast<const uint16_t *>(a->key);
    p.value = static_cast<const uint16_t *>(a->value);
    p.q_stride = a->q_stride;
    p.q_out_stride = a->q_out_stride;
    p.key_stride = a->key_stride;
    p.value_stride = a->value_stride;
    p.query_start_loc = a->query_start_loc;
    p.num_computed = a->num_computed_tokens;
    p.block_table = a->block_table;
    p.key_cache = a->key_cache;
    p.value_cache = a->value_cache;
    p.key_scales = a->key_scales;
    p.value_scales = a->value_scales;
    p.err = a->device_error_word;
    p.k_scale = a->k_scale;
    p.v_scale = a->v_scale;
    p.num_reqs = a->num_reqs;
    p.num_tokens = a->num_tokens;
    p.num_heads_q = a->num_heads_q;
    p.num_heads_kv = a->num_heads_kv;
    p.num_blocks = a->num_blocks;
    p.max_blocks = a->max_blocks_per_req;
    const RopeParams none{};
    return launch_append(a->head_dim, kind, rope ? rope->params : none, p, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? PA_OK
               : PA_ERR_CUDA;
}

}  // extern "C"
