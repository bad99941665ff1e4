// Rotary positions, and the append of new keys and values to a paged cache
// with the rotation on the way.
//
// The rotation of pair i of a row at position p by the angle a = p * f_i:
//   (x, y) -> mag * (x cos a - y sin a,  y cos a + x sin a).
// Angles of far positions are exact to 2^-32 of a turn without 64-bit floating
// point: the planner gives f_i as a fraction of a turn in 64-bit fixed point, so
// p * step_i wraps to the fraction of a turn by itself, and its top 32 bits go
// to sincospif.  cos and sin of the tokens of a CTA are computed once into
// shared memory and used by all of its heads.  Arithmetic in fp32, one
// rounding at the end.
#include "dev.cuh"

namespace pa {
namespace {

using namespace dev;

constexpr int kThreads = 256;

__device__ __forceinline__ void cos_sin(uint64_t step, int32_t pos, float mag, float &c, float &s) {
    const uint64_t turn = static_cast<uint64_t>(static_cast<int64_t>(pos)) * step;
    const float half_turns = static_cast<float>(static_cast<int32_t>(turn >> 32)) * 0x1p-31f;
    sincospif(half_turns, &s, &c);
    c *= mag;
    s *= mag;
}

// cos and sin of `n` tokens: tab[j * rd + i] = cos, tab[j * rd + rd / 2 + i] = sin
// of pair i at the position of token j.
template <typename PosOf>
__device__ __forceinline__ void fill_table(float *tab, const RopeParams &rope, int n, PosOf pos_of) {
    const int half = rope.rotary_dim / 2;
    for (int e = threadIdx.x; e < n * half; e += kThreads) {
        const int j = e / half, i = e - j * half;
        float c, s;
        cos_sin(rope.step[i], pos_of(j), rope.mag, c, s);
        tab[j * rope.rotary_dim + i] = c;
        tab[j * rope.rotary_dim + half + i] = s;
    }
}

// A unit is eight elements of a row that one thread handles, as two groups of
// four at element offsets a and b.  Half layout: dims 4u.. and their partners
// rd / 2 + 4u..; interleaved and pass-through: dims 8u .. 8u + 7.
struct Unit {
    int a, b;       // element offsets
    int freq;       // first of its four pairs; < 0: passes through
    bool inter;
    __device__ __forceinline__ explicit Unit(int u) : a(8 * u), b(8 * u + 4), freq(-1), inter(false) {}
    __device__ __forceinline__ Unit(int u, const RopeParams &r) {
        inter = r.interleaved != 0;
        if (8 * u < r.rotary_dim) {
            freq = 4 * u;
            a = inter ? 8 * u : 4 * u;
            b = inter ? 8 * u + 4 : r.rotary_dim / 2 + 4 * u;
        } else {
            freq = -1;
            a = 8 * u;
            b = 8 * u + 4;
        }
    }
};

__device__ __forceinline__ void unpack4(uint2 w, float (&x)[4]) {
    x[0] = bf16_lo(w.x); x[1] = bf16_hi(w.x); x[2] = bf16_lo(w.y); x[3] = bf16_hi(w.y);
}

// xa, xb: the unit's two groups; tab: its token's table row.  A product and an
// fma: two roundings in 32 bits.
__device__ __forceinline__ void rotate(const Unit &u, const float *tab, int half, float (&xa)[4], float (&xb)[4]) {
    if (u.freq < 0) return;
    const float4 c4 = *reinterpret_cast<const float4 *>(tab + u.freq);
    const float4 s4 = *reinterpret_cast<const float4 *>(tab + half + u.freq);
    const float c[4] = {c4.x, c4.y, c4.z, c4.w}, s[4] = {s4.x, s4.y, s4.z, s4.w};
    auto turn = [](float &x, float &y, float cc, float ss) {
        const float nx = fmaf(x, cc, -(y * ss)), ny = fmaf(y, cc, x * ss);
        x = nx;
        y = ny;
    };
    if (u.inter) {
        turn(xa[0], xa[1], c[0], s[0]);
        turn(xa[2], xa[3], c[1], s[1]);
        turn(xb[0], xb[1], c[2], s[2]);
        turn(xb[2], xb[3], c[3], s[3]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) turn(xa[i], xb[i], c[i], s[i]);
    }
}

// Rotate `n_tok` x `n_heads` rows of bf16 (x and out: first row of the first
// token; consecutive heads D apart) by the table of the tokens.
__device__ __forceinline__ void rotate_rows(const float *tab, const RopeParams &rope, const uint16_t *x, int64_t x_stride,
                                            uint16_t *out, int64_t out_stride, int n_tok, int n_heads, int head_dim) {
    const int upr = head_dim / 8;                   // units per row
    const int rpi = kThreads / upr;                 // rows of one pass over the threads
    const int first = threadIdx.x / upr;
    if (first >= rpi) return;                       // head_dim does not divide the threads' elements
    const Unit u(threadIdx.x % upr, rope);
    const int half = rope.rotary_dim / 2;
    const int rows = n_tok * n_heads;
#pragma unroll 4
    for (int r = first; r < rows; r += rpi) {
        const int j = r / n_heads, h = r - j * n_heads;
        const uint16_t *src = x + j * x_stride + h * head_dim;
        uint16_t *dst = out + j * out_stride + h * head_dim;
        float xa[4], xb[4];
        unpack4(*reinterpret_cast<const uint2 *>(src + u.a), xa);
        unpack4(*reinterpret_cast<const uint2 *>(src + u.b), xb);
        rotate(u, tab + j * rope.rotary_dim, half, xa, xb);
        *reinterpret_cast<uint2 *>(dst + u.a) = make_uint2(pack_bf16x2(xa[0], xa[1]), pack_bf16x2(xa[2], xa[3]));
        *reinterpret_cast<uint2 *>(dst + u.b) = make_uint2(pack_bf16x2(xb[0], xb[1]), pack_bf16x2(xb[2], xb[3]));
    }
}

__global__ void __launch_bounds__(kThreads) rotary_kernel(const __grid_constant__ RopeParams rope, const RotaryParams p) {
    extern __shared__ float4 smem4[];
    float *tab = reinterpret_cast<float *>(smem4);
    grid_launch_dependents();
    grid_dep_wait();
    const int t0 = blockIdx.x * p.tokens_per_cta, h0 = blockIdx.y * p.heads_per_cta;
    const int n = min(p.tokens_per_cta, p.num_tokens - t0), nh = min(p.heads_per_cta, p.num_heads - h0);
    fill_table(tab, rope, n, [&](int j) { return __ldg(p.positions + t0 + j); });
    __syncthreads();
    rotate_rows(tab, rope, p.x + t0 * p.x_stride + h0 * p.head_dim, p.x_stride,
                p.out + t0 * p.out_stride + h0 * p.head_dim, p.out_stride, n, nh, p.head_dim);
}

// ------------------------------------------------------------------ append --
// One segment: the new tokens of one request that lie in one cache block.
struct Segment {
    int32_t t0;      // first token row
    int32_t n;       // tokens (0: nothing to do)
    int32_t pos;     // position of the first token
    int32_t block;   // cache block
};

// Segment `id` of the step.  Request r owns the ids from
// floor(query_start_loc[r] / 16) + 2 r on, which are as many as it can have
// segments (a request of q tokens spans at most floor(q / 16) + 2 blocks), so
// that a grid of num_tokens / 16 + 2 num_reqs CTAs covers every step without
// the lengths being known on the host.  The request is found by a search with
// 32 probes a step, one per lane.  Every warp of a CTA makes the same search.
__device__ __forceinline__ Segment find_segment(const AppendParams &p, int id, bool report) {
    const int lane = threadIdx.x & 31;
    Segment s{0, 0, 0, 0};
    int lo = 0, len = p.num_reqs;   // the last r in [lo, lo + len) whose first id is <= id (r = lo always is)
    while (len > 1) {
        const int step = (len + 31) / 32;
        const int r = lo + lane * step;
        const bool le = lane * step < len && p.query_start_loc[r] / kBlockSize + 2 * r <= id;
        const int k = 31 - __clz(__ballot_sync(0xffffffffu, le) | 1u);
        len = min(step, len - k * step);
        lo += k * step;
    }
    const int qb = p.query_start_loc[lo], qe = min(p.query_start_loc[lo + 1], p.num_tokens);
    const int nc = p.num_computed[lo];
    const int k = id - (qb / kBlockSize + 2 * lo);
    const int off = nc % kBlockSize;
    const int i0 = k == 0 ? 0 : k * kBlockSize - off;   // first token of the segment within the request
    if (qb < 0 || nc < 0 || k < 0 || i0 >= qe - qb) return s;
    s.pos = nc + i0;
    const int page = s.pos / kBlockSize;
    s.block = page < p.max_blocks ? p.block_table[static_cast<int64_t>(lo) * p.max_blocks + page] : -1;
    if (s.block < 0 || s.block >= p.num_blocks) {
        if (report && threadIdx.x == 0 && p.err != nullptr) atomicOr(p.err, kErrBlockRange);
        s.block = -1;                                   // q is still rotated
    }
    s.t0 = qb + i0;
    s.n = min(kBlockSize - s.pos % kBlockSize, qe - qb - i0);
    return s;
}

// Four values in units of the scale -> four codes (lowest byte first): to
// nearest, ties to even, saturating.
template <bool INT8>
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d) {
    if constexpr (INT8) {
        auto one = [](float x) { return static_cast<uint32_t>(__float2int_rn(fminf(fmaxf(x, -127.f), 127.f))) & 0xFFu; };
        return one(a) | one(b) << 8 | one(c) << 16 | one(d) << 24;
    } else {
        return static_cast<uint32_t>(pack_e4m3x2(a, b)) | static_cast<uint32_t>(pack_e4m3x2(c, d)) << 16;
    }
}

template <bool INT8>
__device__ __forceinline__ void decode4(uint32_t w, float (&x)[4]) {
    if constexpr (INT8) {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = static_cast<float>(static_cast<int8_t>(w >> (8 * i)));
    } else {
        uint32_t lo, hi;
        e4m3x4_to_f16x2x2(w, lo, hi);
        x[0] = f16_lo(lo); x[1] = f16_hi(lo); x[2] = f16_lo(hi); x[3] = f16_hi(hi);
    }
}

// The smallest power of two (2^-64 at least) whose qmax-fold reaches amax
// (qmax = 1.75 * 2^8 for E4M3, 127 / 64 * 2^6 for int8).  Powers of two: a
// block's scale then depends on its largest value only, not on the order of
// the appends, a row divided by it is exact before the one rounding to a code,
// and when it grows, the earlier codes are rounded to half the steps or fewer,
// so that their error stays below one step however often it grows.
template <bool INT8>
__device__ __forceinline__ float power_scale(float amax) {
    const uint32_t bits = __float_as_uint(amax);
    const int e = static_cast<int>(bits >> 23) - 127 - (INT8 ? 6 : 8) +
                  ((bits & 0x7FFFFFu) > (INT8 ? 0x7E0000u : 0x600000u) ? 1 : 0);
    return __uint_as_float(static_cast<uint32_t>(max(e, -64) + 127) << 23);
}

// One head's rows of a segment in registers: lane (rsub, u) holds unit u of
// rows it * RPI + rsub as fp32.
template <int D>
struct HeadRows {
    static constexpr int UPR = D / 8, RPI = 32 / UPR, NIT = kBlockSize / RPI;
    float a[NIT][4], b[NIT][4];
};

// Codes of one head's new rows into block-scaled caches, with the block's new
// scale; earlier rows of the block are re-coded when it grows.
template <int D, bool INT8>
__device__ __forceinline__ void store_scaled(const HeadRows<D> &x, const Unit &u, uint8_t *block, int64_t row_stride,
                                             float *scale_at, float old, int first, int n, int lane) {
    using H = HeadRows<D>;
    float amax = 0.f;
    bool nan = false;
#pragma unroll
    for (int it = 0; it < H::NIT; ++it)
#pragma unroll
        for (int i = 0; i < 4; ++i) {   // rows past n hold zeros
            const float va = fabsf(x.a[it][i]), vb = fabsf(x.b[it][i]);
            // infinities saturate and do not count
            amax = fmaxf(amax, va <= 3.4028234663852886e38f ? va : 0.f);
            amax = fmaxf(amax, vb <= 3.4028234663852886e38f ? vb : 0.f);
            if (INT8) nan |= va != va || vb != vb;
        }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    float scale = power_scale<INT8>(amax);
    if (INT8 && __any_sync(0xffffffffu, nan)) scale = __uint_as_float(0x7FC00000u);   // int8 has no NaN: the block's scale is
    if (first > 0 && !(scale != scale)) scale = old != old ? old : fmaxf(old, scale);
    if (lane == 0 && (first == 0 || scale != old)) *scale_at = scale;
    const int rsub = lane / H::UPR, unit = lane % H::UPR;
    if (first > 0 && scale > old) {
        const float ratio = __fdiv_rn(old, scale);
        for (int r = rsub; r < first; r += H::RPI) {
            uint2 *at = reinterpret_cast<uint2 *>(block + r * row_stride + 8 * unit);
            const uint2 w = *at;
            float y[4], z[4];
            decode4<INT8>(w.x, y);
            decode4<INT8>(w.y, z);
            *at = make_uint2(encode4<INT8>(y[0] * ratio, y[1] * ratio, y[2] * ratio, y[3] * ratio),
                             encode4<INT8>(z[0] * ratio, z[1] * ratio, z[2] * ratio, z[3] * ratio));
        }
    }
    // x / scale; by the reciprocal when it is exact (a power of two)
    const bool exact = (__float_as_uint(scale) & 0x7FFFFFu) == 0;
    const float inv = __fdiv_rn(1.f, scale);
    auto q = [&](float v) { return exact ? v * inv : __fdiv_rn(v, scale); };
#pragma unroll
    for (int it = 0; it < H::NIT; ++it) {
        const int r = it * H::RPI + rsub;
        if (r >= n) continue;
        uint8_t *row = block + (first + r) * row_stride;
        *reinterpret_cast<uint32_t *>(row + u.a) = encode4<INT8>(q(x.a[it][0]), q(x.a[it][1]), q(x.a[it][2]), q(x.a[it][3]));
        *reinterpret_cast<uint32_t *>(row + u.b) = encode4<INT8>(q(x.b[it][0]), q(x.b[it][1]), q(x.b[it][2]), q(x.b[it][3]));
    }
}

template <int D, int KIND>
__global__ void __launch_bounds__(kThreads) append_kernel(const __grid_constant__ RopeParams rope, const AppendParams p) {
    using H = HeadRows<D>;
    constexpr bool BLOCK_SCALED = KIND == kCacheE4m3Block || KIND == kCacheInt8Block;
    __shared__ float4 smem4[kBlockSize * D / 4];
    float *tab = reinterpret_cast<float *>(smem4);
    grid_launch_dependents();
    grid_dep_wait();
    const int kv_parts = (p.num_heads_kv + 7) / 8;
    const bool kv = static_cast<int>(blockIdx.y) < kv_parts;
    const Segment s = find_segment(p, blockIdx.x, blockIdx.y == 0);
    if (s.n == 0) return;
    const int half = rope.rotary_dim / 2;
    if (!kv) {
        fill_table(tab, rope, s.n, [&](int j) { return s.pos + j; });
        __syncthreads();
        const int h0 = (static_cast<int>(blockIdx.y) - kv_parts) * p.q_heads_per_cta;
        rotate_rows(tab, rope, p.q + s.t0 * p.q_stride + h0 * D, p.q_stride, p.q_out + s.t0 * p.q_out_stride + h0 * D,
                    p.q_out_stride, s.n, min(p.q_heads_per_cta, p.num_heads_q - h0), D);
        return;
    }
    if (s.block < 0) return;
    const int lane = threadIdx.x & 31;
    const int h = blockIdx.y * 8 + threadIdx.x / 32;
    const bool mine = h < p.num_heads_kv;
    const int rsub = lane / H::UPR;
    const Unit u(lane % H::UPR, rope);
    const Unit uv(lane % H::UPR);   // values: eight consecutive dims
    const int first = s.pos % kBlockSize;
    // every row's loads before the first use
    uint2 ka[H::NIT], kb[H::NIT];
    uint4 v[H::NIT];
    float old_k = 0.f, old_v = 0.f;
    if (mine) {
        const int64_t at = static_cast<int64_t>(s.block) * p.num_heads_kv + h;
        if (BLOCK_SCALED && first > 0) {
            old_k = p.key_scales[at];
            old_v = p.value_scales[at];
        }
#pragma unroll
        for (int it = 0; it < H::NIT; ++it) {
            const int r = it * H::RPI + rsub;
            ka[it] = kb[it] = make_uint2(0, 0);
            v[it] = make_uint4(0, 0, 0, 0);
            if (r < s.n) {
                const uint16_t *k = p.key + (s.t0 + r) * p.key_stride + h * D;
                ka[it] = *reinterpret_cast<const uint2 *>(k + u.a);
                kb[it] = *reinterpret_cast<const uint2 *>(k + u.b);
                v[it] = *reinterpret_cast<const uint4 *>(p.value + (s.t0 + r) * p.value_stride + h * D + uv.a);
            }
        }
    }
    if (half > 0) fill_table(tab, rope, s.n, [&](int j) { return s.pos + j; });
    __syncthreads();
    if (!mine) return;
    const int64_t row_stride = static_cast<int64_t>(p.num_heads_kv) * D;
    const int64_t base = static_cast<int64_t>(s.block) * kBlockSize * row_stride + h * D;   // element of row 0
    if constexpr (BLOCK_SCALED) {
        const int64_t at = static_cast<int64_t>(s.block) * p.num_heads_kv + h;
        H x;
#pragma unroll
        for (int it = 0; it < H::NIT; ++it) {
            unpack4(ka[it], x.a[it]);
            unpack4(kb[it], x.b[it]);
            if (it * H::RPI + rsub < s.n) rotate(u, tab + (it * H::RPI + rsub) * rope.rotary_dim, half, x.a[it], x.b[it]);
        }
        store_scaled<D, KIND == kCacheInt8Block>(x, u, static_cast<uint8_t *>(p.key_cache) + base, row_stride,
                                                 p.key_scales + at, old_k, first, s.n, lane);
#pragma unroll
        for (int it = 0; it < H::NIT; ++it) {
            unpack4(make_uint2(v[it].x, v[it].y), x.a[it]);
            unpack4(make_uint2(v[it].z, v[it].w), x.b[it]);
        }
        store_scaled<D, KIND == kCacheInt8Block>(x, uv, static_cast<uint8_t *>(p.value_cache) + base, row_stride,
                                                 p.value_scales + at, old_v, first, s.n, lane);
    } else {
#pragma unroll
        for (int it = 0; it < H::NIT; ++it) {
            const int r = it * H::RPI + rsub;
            if (r >= s.n) continue;
            float xa[4], xb[4];
            unpack4(ka[it], xa);
            unpack4(kb[it], xb);
            rotate(u, tab + r * rope.rotary_dim, half, xa, xb);
            const int64_t row = base + (first + r) * row_stride;
            if constexpr (KIND == kCacheBf16) {
                uint16_t *k = static_cast<uint16_t *>(p.key_cache) + row;
                if (half > 0) {
                    ka[it] = make_uint2(pack_bf16x2(xa[0], xa[1]), pack_bf16x2(xa[2], xa[3]));
                    kb[it] = make_uint2(pack_bf16x2(xb[0], xb[1]), pack_bf16x2(xb[2], xb[3]));
                }   // else a bit copy (a NaN keeps its bits)
                *reinterpret_cast<uint2 *>(k + u.a) = ka[it];
                *reinterpret_cast<uint2 *>(k + u.b) = kb[it];
                *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.value_cache) + row + uv.a) = v[it];
            } else {
                // codes of x / k_scale, the quotient rounded in 32 bits as pa_write_kv_fp8 does
                uint8_t *k = static_cast<uint8_t *>(p.key_cache) + row;
                auto q = [&](float y) { return __fdiv_rn(y, p.k_scale); };
                *reinterpret_cast<uint32_t *>(k + u.a) = encode4<false>(q(xa[0]), q(xa[1]), q(xa[2]), q(xa[3]));
                *reinterpret_cast<uint32_t *>(k + u.b) = encode4<false>(q(xb[0]), q(xb[1]), q(xb[2]), q(xb[3]));
                *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(p.value_cache) + row + uv.a) =
                    e4m3_quantize8(v[it], p.v_scale);
            }
        }
    }
}

template <int D>
cudaError_t launch_append_d(int kind, const RopeParams &rope, const AppendParams &p, dim3 grid, cudaStream_t stream) {
    switch (kind) {
        case kCacheBf16: return launch_pdl(append_kernel<D, kCacheBf16>, grid, dim3(kThreads), 0, stream, rope, p);
        case kCacheE4m3: return launch_pdl(append_kernel<D, kCacheE4m3>, grid, dim3(kThreads), 0, stream, rope, p);
        case kCacheE4m3Block:
            return launch_pdl(append_kernel<D, kCacheE4m3Block>, grid, dim3(kThreads), 0, stream, rope, p);
        case kCacheInt8Block:
            return launch_pdl(append_kernel<D, kCacheInt8Block>, grid, dim3(kThreads), 0, stream, rope, p);
    }
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_rotary(const RopeParams &rope, const RotaryParams &p0, cudaStream_t stream) {
    RotaryParams p = p0;
    if (p.num_tokens <= 0) return cudaSuccess;
    p.tokens_per_cta = p.num_tokens > 2048 ? 16 : p.num_tokens > 512 ? 4 : 1;
    p.heads_per_cta = p.num_heads < 16 ? p.num_heads : 16;
    const dim3 grid((p.num_tokens + p.tokens_per_cta - 1) / p.tokens_per_cta,
                    (p.num_heads + p.heads_per_cta - 1) / p.heads_per_cta);
    return launch_pdl(rotary_kernel, grid, dim3(kThreads), sizeof(float) * p.tokens_per_cta * rope.rotary_dim, stream, rope, p);
}

cudaError_t launch_append(int head_dim, int kind, const RopeParams &rope, const AppendParams &p0, cudaStream_t stream) {
    AppendParams p = p0;
    if (p.num_tokens <= 0 || p.num_reqs <= 0) return cudaSuccess;
    p.q_heads_per_cta = p.num_heads_q < 16 ? p.num_heads_q : 16;
    const int q_parts = p.q == nullptr ? 0 : (p.num_heads_q + p.q_heads_per_cta - 1) / p.q_heads_per_cta;
    const dim3 grid(p.num_tokens / kBlockSize + 2 * p.num_reqs, (p.num_heads_kv + 7) / 8 + q_parts);
    if (head_dim == 128) return launch_append_d<128>(kind, rope, p, grid, stream);
    if (head_dim == 64) return launch_append_d<64>(kind, rope, p, grid, stream);
    return cudaErrorInvalidValue;
}

}  // namespace pa
