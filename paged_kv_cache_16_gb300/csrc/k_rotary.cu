// Rotary positions, and the append of new keys and values to a paged cache
// with the rotation on the way.
//
// The rotation of pair i of a row at position p by the angle a = p * f_i:
//   (x, y) -> mag * (x cos a - y sin a,  y cos a + x sin a).
// Angles of far positions are exact to 2^-32 of a turn without 64-bit floating
// point: the planner gives f_i as a fraction of a turn in 64-bit fixed point, so
// p * step_i wraps to the fraction of a turn by itself, whose top 32 bits are used:
// 24 of them through sincospif, the rest as a turn of the result by that little
// (without it the angle is off by up to 2^-26 of a turn: 9.4e-8, more than the
// rounding of cos and sin).  cos and sin of the tokens of a CTA are computed once into
// shared memory and used by all of its heads.  Arithmetic in fp32, one
// rounding at the end.
//
// With positions on several axes (time, height, width) pair i turns by
// p_axis(i) * f_i: the table is made from as many positions per token, a thread of
// it keeps one pair and so one axis, and nothing else differs (8192 tokens x 40 heads
// 27.1 us instead of 26.7; 64 tokens 2.1 us; the append of four chunks of 2048 into bf16
// caches 32.9 instead of 31.8).
#include "dev.cuh"

namespace pa {
namespace {

using namespace dev;

constexpr int kThreads = 256;

__device__ __forceinline__ void cos_sin(uint64_t step, int32_t pos, float mag, float &c, float &s) {
    const uint64_t turn = static_cast<uint64_t>(static_cast<int64_t>(pos)) * step;
    const int32_t t = static_cast<int32_t>((turn + 0x80000000u) >> 32);   // of 2^-31 half a turn, to nearest
    const float head = __int2float_rz(t);                 // (towards 0: exact on the way back)
    sincospif(head * 0x1p-31f, &s, &c);
    const float rest = static_cast<float>(t - static_cast<int32_t>(head)) * 1.462918079e-9f;   // pi 2^-31
    const float c1 = fmaf(-rest, s, c), s1 = fmaf(rest, c, s);
    c = c1 * mag;
    s = s1 * mag;
}

// cos and sin of `n` tokens: tab[j * rd + i] = cos, tab[j * rd + rd / 2 + i] = sin
// of pair i at the position of token j.  A thread keeps one pair, whose step it
// reads once, through the generic address of the kernel's argument: 32 lanes in
// one access, where constant loads of 32 addresses go one by one (a constant load
// per entry: 64 tokens 2.2 us instead of 1.8, 8192 tokens x 8 heads 10.4 instead of
// 7.6, an append of two chunks 19.6 instead of 18.5; once per thread, 2.0 and 18.4,
// but a decode step's append 3.6 instead of 3.5).
template <bool AXES>
struct RopeArg_ { using type = RopeParams; };
template <>
struct RopeArg_<true> { using type = AxesRopeParams; };
template <bool AXES>
using RopeArg = typename RopeArg_<AXES>::type;

template <bool AXES>
struct TableMaker {
    int i, j0, tokens;   // pair, first token, tokens a pass (0: no part of the table)
    int axis;            // of its positions
    uint64_t step;
    __device__ __forceinline__ TableMaker(const RopeArg<AXES> &rope, int n) : i(0), j0(0), tokens(0), axis(0), step(0) {
        const int half = rope.rotary_dim / 2;
        if (half == 0) return;
        j0 = static_cast<int>(threadIdx.x) / half;
        i = static_cast<int>(threadIdx.x) - j0 * half;
        tokens = kThreads / half;
        const uint64_t *steps;   // (opaque, or the load would be a constant one)
        asm("mov.u64 %0, %1;" : "=l"(steps) : "l"(rope.step));
        if (j0 < min(tokens, n)) step = steps[i];
        if constexpr (AXES) {
            const uint8_t *axes;
            asm("mov.u64 %0, %1;" : "=l"(axes) : "l"(rope.axis));
            if (j0 < min(tokens, n)) axis = axes[i];
        }
    }
    template <typename PosOf>
    __device__ __forceinline__ void fill(float *tab, const RopeParams &rope, int n, PosOf pos_of) const {
        if (j0 >= tokens) return;
        float *at = tab + j0 * rope.rotary_dim + i;
        for (int j = j0; j < n; j += tokens, at += tokens * rope.rotary_dim) {
            float c, s;
            cos_sin(step, pos_of(j, axis), rope.mag, c, s);
            at[0] = c;
            at[rope.rotary_dim / 2] = s;
        }
    }
};

// A unit is 2 W elements of a row that one thread handles, as two groups of W
// (8 or 16 bytes) at element offsets a and b.  Half layout: dims W u.. and their
// partners rd / 2 + W u..; interleaved and pass-through: dims 2 W u .. + 2 W - 1.
// W = 8 where rotary_dim and head_dim are multiples of 16, else 4.
template <int W>
struct Unit {
    int a, b;       // element offsets
    int freq;       // first of its W pairs; < 0: passes through
    bool inter;
    __device__ __forceinline__ explicit Unit(int u) : a(2 * W * u), b(2 * W * u + W), freq(-1), inter(false) {}
    __device__ __forceinline__ Unit(int u, const RopeParams &r) : Unit(u) {
        if (2 * W * u >= r.rotary_dim) return;
        freq = W * u;
        inter = r.interleaved != 0;
        if (!inter) {
            a = W * u;
            b = r.rotary_dim / 2 + W * u;
        }
    }
};

template <int W>
struct Raw {   // W bf16
    uint32_t w[W / 2];
};

template <int W>
__device__ __forceinline__ Raw<W> load_raw(const uint16_t *p) {
    Raw<W> r;
    if constexpr (W == 8) {
        const uint4 v = *reinterpret_cast<const uint4 *>(p);
        r.w[0] = v.x; r.w[1] = v.y; r.w[2] = v.z; r.w[3] = v.w;
    } else {
        const uint2 v = *reinterpret_cast<const uint2 *>(p);
        r.w[0] = v.x; r.w[1] = v.y;
    }
    return r;
}

template <int W>
__device__ __forceinline__ void store_raw(uint16_t *p, const Raw<W> &r) {
    if constexpr (W == 8) *reinterpret_cast<uint4 *>(p) = make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
    else *reinterpret_cast<uint2 *>(p) = make_uint2(r.w[0], r.w[1]);
}

template <int W>
__device__ __forceinline__ void unpack(const Raw<W> &r, float (&x)[W]) {
#pragma unroll
    for (int i = 0; i < W / 2; ++i) {
        x[2 * i] = bf16_lo(r.w[i]);
        x[2 * i + 1] = bf16_hi(r.w[i]);
    }
}

template <int W>
__device__ __forceinline__ Raw<W> pack(const float (&x)[W]) {
    Raw<W> r;
#pragma unroll
    for (int i = 0; i < W / 2; ++i) r.w[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
    return r;
}

// cos and sin of a unit's pairs at one token's position
template <int W>
struct Turn {
    float c[W], s[W];
    __device__ __forceinline__ void load(const Unit<W> &u, const float *tab, int half) {
        if (u.freq < 0) return;
#pragma unroll
        for (int i = 0; i < W; i += 4) {
            const float4 c4 = *reinterpret_cast<const float4 *>(tab + u.freq + i);
            const float4 s4 = *reinterpret_cast<const float4 *>(tab + half + u.freq + i);
            c[i] = c4.x; c[i + 1] = c4.y; c[i + 2] = c4.z; c[i + 3] = c4.w;
            s[i] = s4.x; s[i + 1] = s4.y; s[i + 2] = s4.z; s[i + 3] = s4.w;
        }
    }
    // a product and an fma: two roundings in 32 bits
    __device__ __forceinline__ void apply(const Unit<W> &u, float (&xa)[W], float (&xb)[W]) const {
        if (u.freq < 0) return;
        auto turn = [](float &x, float &y, float cc, float ss) {
            const float nx = fmaf(x, cc, -(y * ss)), ny = fmaf(y, cc, x * ss);
            x = nx;
            y = ny;
        };
        if (u.inter) {
#pragma unroll
            for (int i = 0; i < W / 2; ++i) {
                turn(xa[2 * i], xa[2 * i + 1], c[i], s[i]);
                turn(xb[2 * i], xb[2 * i + 1], c[W / 2 + i], s[W / 2 + i]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < W; ++i) turn(xa[i], xb[i], c[i], s[i]);
        }
    }
};

// Rotate `n_tok` x `n_heads` rows of bf16 (x and out: first row of the first
// token; consecutive heads D apart) by the table of the tokens.  The threads are
// dealt to 1 << log_tokens >= n_tok tokens; a thread keeps one unit of one
// token, its cos and sin in registers, and walks the heads with kBatch rows'
// loads before the first of their stores.
template <int W, int kBatch>
__device__ __forceinline__ void rotate_rows(const float *tab, const RopeParams &rope, const uint16_t *x, int64_t x_stride,
                                            uint16_t *out, int64_t out_stride, int n_tok, int log_tokens, int n_heads,
                                            int head_dim) {
    const int per = kThreads >> log_tokens;         // threads of a token
    const int j = threadIdx.x / per, r = threadIdx.x % per;
    const int upr = head_dim / (2 * W);             // units per row
    const int lanes = per / upr;                    // rows at a time
    const int h0 = r / upr;
    if (j >= n_tok || h0 >= lanes) return;
    const Unit<W> u(r % upr, rope);
    Turn<W> turn;
    turn.load(u, tab + j * rope.rotary_dim, rope.rotary_dim / 2);
    x += j * x_stride;
    out += j * out_stride;
    for (int h = h0; h < n_heads; h += kBatch * lanes) {
        Raw<W> wa[kBatch], wb[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int hk = h + k * lanes;
            if (hk < n_heads) {
                wa[k] = load_raw<W>(x + hk * head_dim + u.a);
                wb[k] = load_raw<W>(x + hk * head_dim + u.b);
            }
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int hk = h + k * lanes;
            if (hk >= n_heads) break;
            float xa[W], xb[W];
            unpack<W>(wa[k], xa);
            unpack<W>(wb[k], xb);
            turn.apply(u, xa, xb);
            store_raw<W>(out + hk * head_dim + u.a, pack<W>(xa));
            store_raw<W>(out + hk * head_dim + u.b, pack<W>(xb));
        }
    }
}

// Bound by HBM (8192 tokens x 40 heads of 128: 26.5 us, 6.3 TB/s; 43.3 us with
// cos and sin read from shared memory per row, 8-byte pieces and one row of a thread
// in flight) and by the launch for a decode step (64 tokens: 1.8 us).  A CTA's rows
// are asked into L2 before its table of cos and sin is made, from 1 MB of rows on
// (28.8 us without; 512 tokens 3.2 and 3.7, 128 tokens 2.35 and 2.5, 64 tokens the
// same; 1021 tokens x 7 heads of 64 1.76 and 1.65).
template <int W, bool AXES>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const __grid_constant__ RopeArg<AXES> rope, const RotaryParams p) {
    extern __shared__ float4 smem4[];
    float *tab = reinterpret_cast<float *>(smem4);
    grid_launch_dependents();
    const int t0 = blockIdx.x << p.log_tokens, h0 = blockIdx.y * p.heads_per_cta;
    const int n = min(1 << p.log_tokens, p.num_tokens - t0), nh = min(p.heads_per_cta, p.num_heads - h0);
    const TableMaker<AXES> table(rope, n);
    grid_dep_wait();
    if (W == 8 && p.prefetch && static_cast<int>(threadIdx.x) < n)   // (16-byte pieces: aligned rows)
        bulk_prefetch_l2(p.x + (t0 + static_cast<int>(threadIdx.x)) * p.x_stride + h0 * p.head_dim, nh * p.head_dim * 2);
    table.fill(tab, rope, n, [&](int j, int axis) { return __ldg(p.positions + (AXES ? axis * p.axis_stride : 0) + t0 + j); });
    __syncthreads();
    rotate_rows<W, W == 8 ? 5 : 8>(tab, rope, p.x + t0 * p.x_stride + h0 * p.head_dim, p.x_stride,
                   p.out + t0 * p.out_stride + h0 * p.head_dim, p.out_stride, n, p.log_tokens, nh, p.head_dim);
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
// the lengths being known on the host.  Every warp of a CTA makes the same
// search: 32 probes a step, one per lane, while there are more than 128 requests
// left, then the starts and lengths of all of them at once, so that two
// dependent loads (these, the block id) stand before the scales and the stores.
__device__ __forceinline__ Segment find_segment(const AppendParams &p, int id) {
    const int lane = threadIdx.x & 31;
    Segment s{0, 0, 0, 0};
    // the last request in [lo, lo + len) whose first id is <= id (lo always is)
    int lo = 0, len = p.num_reqs;
    while (len > 128) {
        const int step = (len + 31) / 32;
        const int r = lo + lane * step;
        const bool le = lane * step < len && p.query_start_loc[r] / kBlockSize + 2 * r <= id;
        const int k = 31 - __clz(__ballot_sync(0xffffffffu, le) | 1u);
        len = min(step, len - k * step);
        lo += k * step;
    }
    // up to 128 requests: all their starts and lengths in one round of loads, lane
    // l holding requests lo + l + 32 k
    int32_t qs[4], cs[4], last = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int i = lane + 32 * k;
        qs[k] = i < len ? p.query_start_loc[lo + i] : 0;
        cs[k] = i < len ? p.num_computed[lo + i] : 0;
    }
    if (lane == 0) last = p.query_start_loc[lo + len];
    int at = -1;
#pragma unroll
    for (int k = 0; k < 4; ++k)
        at += __popc(__ballot_sync(0xffffffffu, lane + 32 * k < len && qs[k] / kBlockSize + 2 * (lo + lane + 32 * k) <= id));
    at = max(at, 0);
    auto pick = [&](const int32_t (&v)[4], int i) {
        int32_t r = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int32_t y = __shfl_sync(0xffffffffu, v[k], i & 31);
            if (i >> 5 == k) r = y;
        }
        return r;
    };
    const int qb = pick(qs, at), nc = pick(cs, at);
    const int end = __shfl_sync(0xffffffffu, last, 0), next = pick(qs, at + 1);
    const int qe = min(at + 1 < len ? next : end, p.num_tokens);
    lo += at;
    const int k = id - (qb / kBlockSize + 2 * lo);
    const int off = nc % kBlockSize;
    const int i0 = k == 0 ? 0 : k * kBlockSize - off;   // first token of the segment within the request
    if (qb < 0 || nc < 0 || k < 0 || i0 >= qe - qb) return s;
    s.pos = nc + i0;
    s.t0 = qb + i0;
    s.n = min(kBlockSize - s.pos % kBlockSize, qe - qb - i0);
    const int page = s.pos / kBlockSize;
    s.block = page < p.max_blocks ? p.block_table[static_cast<int64_t>(lo) * p.max_blocks + page] : -1;
    return s;
}

// whether the segment's block exists (else reported); first use of the id
__device__ __forceinline__ bool block_ok(const AppendParams &p, const Segment &s, bool report) {
    if (s.block >= 0 && s.block < p.num_blocks) return true;
    if (report && threadIdx.x == 0 && p.err != nullptr) atomicOr(p.err, kErrBlockRange);
    return false;
}

// Four values in units of the scale -> four codes (lowest byte first): to
// nearest, ties to even, saturating.  int8: the sum with 1.5 x 2^23 rounds to a
// whole number, two's complement in its low byte.
template <bool INT8>
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d) {
    if constexpr (INT8) {
        auto one = [](float x) { return __float_as_uint(__fadd_rn(fminf(fmaxf(x, -127.f), 127.f), 12582912.f)); };
        return prmt(prmt(one(a), one(b), 0x0040u), prmt(one(c), one(d), 0x0040u), 0x5410u);
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

// One head's rows of a segment: lane (rsub, u) of its warp holds unit u of rows
// it * RPI + rsub; rows past the segment hold zeros.
template <int D, int W>
struct HeadRows {
    static constexpr int UPR = D / (2 * W), RPI = 32 / UPR, NIT = kBlockSize / RPI;
};

// the largest finite magnitude (infinities saturate and do not count), and
// whether there is a NaN
template <int W>
__device__ __forceinline__ void track(const float (&x)[W], float &amax, bool &nan) {
#pragma unroll
    for (int i = 0; i < W; ++i) {
        const float v = fabsf(x[i]);
        amax = fmaxf(amax, v <= 3.4028234663852886e38f ? v : 0.f);
        nan |= v != v;
    }
}

template <int W>
__device__ __forceinline__ void store_codes(uint8_t *p, const uint32_t (&c)[W / 4]) {
    if constexpr (W == 8) *reinterpret_cast<uint2 *>(p) = make_uint2(c[0], c[1]);
    else *reinterpret_cast<uint32_t *>(p) = c[0];
}

// Codes of one head's new rows into block-scaled caches, with the block's new
// scale; earlier rows of the block are re-coded when it grows.
// rows(it, xa, xb) gives the lane's two groups of row it * RPI + rsub.
template <int D, int W, bool INT8, typename Rows>
__device__ __forceinline__ void store_scaled(Rows rows, float amax, bool nan, const Unit<W> &u, uint8_t *block,
                                             int64_t row_stride, float *scale_at, float old, int first, int n, int lane) {
    using H = HeadRows<D, W>;
    float scale = power_scale<INT8>(amax);
    if (INT8 && nan) scale = __uint_as_float(0x7FC00000u);   // int8 has no NaN: the block's scale is
    if (first > 0 && !(scale != scale)) scale = old != old ? old : fmaxf(old, scale);
    if (lane == 0 && (first == 0 || scale != old)) *scale_at = scale;
    const int rsub = lane / H::UPR, unit = lane % H::UPR;
    if (first > 0 && scale > old) {
        const float ratio = __fdiv_rn(old, scale);
        for (int r = rsub; r < first; r += H::RPI) {
            uint8_t *at = block + r * row_stride + 2 * W * unit;
#pragma unroll
            for (int i = 0; i < W / 4; ++i) {
                uint2 *q = reinterpret_cast<uint2 *>(at) + i;
                const uint2 w = *q;
                float y[4], z[4];
                decode4<INT8>(w.x, y);
                decode4<INT8>(w.y, z);
                *q = make_uint2(encode4<INT8>(y[0] * ratio, y[1] * ratio, y[2] * ratio, y[3] * ratio),
                                encode4<INT8>(z[0] * ratio, z[1] * ratio, z[2] * ratio, z[3] * ratio));
            }
        }
    }
    auto store = [&](auto quotient) {
#pragma unroll
        for (int it = 0; it < H::NIT; ++it) {
            if (it * H::RPI >= n) break;
            const int r = it * H::RPI + rsub;
            float xa[W], xb[W];
            rows(it, xa, xb);
            uint32_t ca[W / 4], cb[W / 4];
#pragma unroll
            for (int i = 0; i < W; ++i) { xa[i] = quotient(xa[i]); xb[i] = quotient(xb[i]); }
#pragma unroll
            for (int i = 0; i < W / 4; ++i) {
                ca[i] = encode4<INT8>(xa[4 * i], xa[4 * i + 1], xa[4 * i + 2], xa[4 * i + 3]);
                cb[i] = encode4<INT8>(xb[4 * i], xb[4 * i + 1], xb[4 * i + 2], xb[4 * i + 3]);
            }
            if (r < n) {
                uint8_t *row = block + (first + r) * row_stride;
                store_codes<W>(row + u.a, ca);
                store_codes<W>(row + u.b, cb);
            }
        }
    };
    // x / scale; by the reciprocal when it is exact (a power of two).  A scale of
    // another writer's goes the slow way, kept out of the unrolled code
    if ((__float_as_uint(scale) & 0x7FFFFFu) == 0) {
        const float inv = __uint_as_float((254u << 23) - __float_as_uint(scale));   // 2^-e of 2^e, |e| < 127
        const bool plain = __float_as_uint(scale) - (1u << 23) < (252u << 23);
        store([inv = plain ? inv : __fdiv_rn(1.f, scale)](float v) { return v * inv; });
    } else {
        store([scale](float v) { return __fdiv_rn(v, scale); });
    }
}

__device__ __forceinline__ int log2_up(int n) { return n <= 1 ? 0 : 32 - __clz(n - 1); }

// Which part of a segment a CTA handles: the queries of up to 32 heads, or keys
// or values of 8 kv heads (one per warp).  The queries, the longest parts, come
// first in the grid.  K and V of a block are independent (each has scales of its
// own): in CTAs of their own the dependent chain of a decode step is shorter
// (64 requests, Hq 32, Hkv 8, int8: 3.6 us against 4.5 with both in one CTA, before
// the table's steps were read in one access; two chunks of 2048 tokens into E4M3
// codes 19.6 against 21.2; four into bf16 31.8 against 30.5).  Now 3.5, 18.5 (4.7
// TB/s; 12.7 us at the copy rate) and 31.6 us (5.8 TB/s): bound by latency below a
// wave of CTAs (a decode step: launch, starts and lengths, block id, scale), by HBM
// above, and by both where the queries' CTAs (~10 us each, two per SM) are followed
// by the last keys and values (~4 us each).  Queries of 8 / 16 / 32 heads per CTA
// 22.9 / 20.2 / 18.5, a segment's parts side by side in the grid 19.2, keys and
// values first with 16 heads 19.3; rows asked into L2 first 19.4.
template <int D, int KIND, int W, bool AXES>
__global__ void __launch_bounds__(kThreads, 2) append_kernel(const __grid_constant__ RopeArg<AXES> rope, const AppendParams p) {
    using H = HeadRows<D, W>;
    constexpr bool BLOCK_SCALED = KIND == kCacheE4m3Block || KIND == kCacheInt8Block;
    constexpr bool INT8 = KIND == kCacheInt8Block;
    __shared__ float4 smem4[kBlockSize * D / 4];
    float *tab = reinterpret_cast<float *>(smem4);
    grid_launch_dependents();
    grid_dep_wait();
    const int kv_parts = (p.num_heads_kv + 7) / 8;
    const int part = (static_cast<int>(blockIdx.y) + 2 * kv_parts) % static_cast<int>(gridDim.y);
    const Segment s = find_segment(p, blockIdx.x);
    if (s.n == 0) return;
    // (axes: a row turns by positions of its own, wherever it goes in the cache)
    auto pos_of = [&](int j, int axis) {
        if constexpr (AXES) return __ldg(p.positions + axis * p.axis_stride + s.t0 + j);
        return s.pos + j;
    };
    if (part >= 2 * kv_parts) {
        TableMaker<AXES>(rope, s.n).fill(tab, rope, s.n, pos_of);
        __syncthreads();
        const int h0 = (part - 2 * kv_parts) * p.q_heads_per_cta;
        rotate_rows<W, 8>(tab, rope, p.q + s.t0 * p.q_stride + h0 * D, p.q_stride, p.q_out + s.t0 * p.q_out_stride + h0 * D,
                          p.q_out_stride, s.n, log2_up(s.n), min(p.q_heads_per_cta, p.num_heads_q - h0), D);
        return;
    }
    const bool value = part >= kv_parts;
    const int half = value ? 0 : rope.rotary_dim / 2;   // > 0: rotate
    const int lane = threadIdx.x & 31;
    const int h = (value ? part - kv_parts : part) * 8 + threadIdx.x / 32;
    const bool mine = h < p.num_heads_kv;
    const int rsub = lane / H::UPR;
    const Unit<W> u = half > 0 ? Unit<W>(lane % H::UPR, rope) : Unit<W>(lane % H::UPR);
    const int first = s.pos % kBlockSize;
    // every row's loads before the first use of the block id
    const uint16_t *src = value ? p.value : p.key;
    const int64_t stride = value ? p.value_stride : p.key_stride;
    Raw<W> ra[H::NIT], rb[H::NIT];
#pragma unroll
    for (int it = 0; it < H::NIT; ++it) {
        const int r = it * H::RPI + rsub;
        ra[it] = rb[it] = Raw<W>{};
        if (mine && r < s.n) {
            const uint16_t *x = src + (s.t0 + r) * stride + h * D;
            ra[it] = load_raw<W>(x + u.a);
            rb[it] = load_raw<W>(x + u.b);
        }
    }
    if (half > 0) TableMaker<AXES>(rope, s.n).fill(tab, rope, s.n, pos_of);
    __syncthreads();
    if (!block_ok(p, s, part == 0) || !mine) return;
    const int64_t row_stride = static_cast<int64_t>(p.num_heads_kv) * D;
    const int64_t base = static_cast<int64_t>(s.block) * kBlockSize * row_stride + h * D;   // element of row 0
    void *cache = value ? p.value_cache : p.key_cache;
    // the lane's two groups of row it * RPI + rsub, rotated (for the maximum and
    // once more for the codes: fewer registers than keeping the rotated rows)
    auto row_of = [&](int it, float (&a)[W], float (&b)[W]) {
        unpack<W>(ra[it], a);
        unpack<W>(rb[it], b);
        if (half == 0) return;
        Turn<W> turn;   // (a row past the segment: of its last token, zeros all the same)
        turn.load(u, tab + min(it * H::RPI + rsub, s.n - 1) * rope.rotary_dim, half);
        turn.apply(u, a, b);
    };
    if constexpr (BLOCK_SCALED) {
        float *scale_at = (value ? p.value_scales : p.key_scales) + static_cast<int64_t>(s.block) * p.num_heads_kv + h;
        const float old = first > 0 ? *scale_at : 0.f;
        float amax = 0.f;
        bool nan = false;
#pragma unroll
        for (int it = 0; it < H::NIT; ++it) {
            if (it * H::RPI >= s.n) break;
            float xa[W], xb[W];
            row_of(it, xa, xb);
            track<W>(xa, amax, nan);
            track<W>(xb, amax, nan);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        if (INT8) nan = __any_sync(0xffffffffu, nan);
        store_scaled<D, W, INT8>(row_of, amax, nan, u, static_cast<uint8_t *>(cache) + base, row_stride, scale_at, old, first,
                                 s.n, lane);
    } else {
#pragma unroll
        for (int it = 0; it < H::NIT; ++it) {
            if (it * H::RPI >= s.n) break;
            const int r = it * H::RPI + rsub;
            float xa[W], xb[W];
            row_of(it, xa, xb);
            if (r >= s.n) continue;
            const int64_t row = base + (first + r) * row_stride;
            if constexpr (KIND == kCacheBf16) {
                uint16_t *c = static_cast<uint16_t *>(cache) + row;
                // (not rotated: a bit copy, a NaN keeps its bits)
                store_raw<W>(c + u.a, half > 0 ? pack<W>(xa) : ra[it]);
                store_raw<W>(c + u.b, half > 0 ? pack<W>(xb) : rb[it]);
            } else {
                // codes of x / scale, the quotient rounded in 32 bits as pa_write_kv_fp8 does
                uint8_t *c = static_cast<uint8_t *>(cache) + row;
                const float scale = value ? p.v_scale : p.k_scale;
                uint32_t ca[W / 4], cb[W / 4];
#pragma unroll
                for (int i = 0; i < W / 4; ++i) {
                    ca[i] = encode4<false>(__fdiv_rn(xa[4 * i], scale), __fdiv_rn(xa[4 * i + 1], scale),
                                           __fdiv_rn(xa[4 * i + 2], scale), __fdiv_rn(xa[4 * i + 3], scale));
                    cb[i] = encode4<false>(__fdiv_rn(xb[4 * i], scale), __fdiv_rn(xb[4 * i + 1], scale),
                                           __fdiv_rn(xb[4 * i + 2], scale), __fdiv_rn(xb[4 * i + 3], scale));
                }
                store_codes<W>(c + u.a, ca);
                store_codes<W>(c + u.b, cb);
            }
        }
    }
}

// units of 2 x 8 elements where every group of a row is 16-byte aligned
bool wide_units(const RopeParams &rope, int head_dim) { return rope.rotary_dim % 16 == 0 && head_dim % 16 == 0; }

template <int D, int W, bool AXES>
cudaError_t launch_append_d(int kind, const RopeArg<AXES> &rope, const AppendParams &p, dim3 grid, cudaStream_t stream) {
    switch (kind) {
        case kCacheBf16: return launch_pdl(append_kernel<D, kCacheBf16, W, AXES>, grid, dim3(kThreads), 0, stream, rope, p);
        case kCacheE4m3: return launch_pdl(append_kernel<D, kCacheE4m3, W, AXES>, grid, dim3(kThreads), 0, stream, rope, p);
        case kCacheE4m3Block:
            return launch_pdl(append_kernel<D, kCacheE4m3Block, W, AXES>, grid, dim3(kThreads), 0, stream, rope, p);
        case kCacheInt8Block:
            return launch_pdl(append_kernel<D, kCacheInt8Block, W, AXES>, grid, dim3(kThreads), 0, stream, rope, p);
    }
    return cudaErrorInvalidValue;
}

template <bool AXES>
cudaError_t launch_rotary_t(const RopeArg<AXES> &rope, const RotaryParams &p0, cudaStream_t stream) {
    RotaryParams p = p0;
    if (p.num_tokens <= 0) return cudaSuccess;
    p.heads_per_cta = p.num_heads < 40 ? p.num_heads : 40;
    // tokens of a CTA: as many as give its threads up to 5 units each, one batch of
    // loads (10 units: 4096 tokens x 40 heads 15.4 us instead of 14.5, 8192 tokens
    // the same), while there is a CTA for every SM and a thread for every unit of a
    // row
    const bool wide = wide_units(rope, p.head_dim);
    const int upr = p.head_dim / (wide ? 16 : 8);
    p.log_tokens = 0;
    while (p.log_tokens < 4 && (p.heads_per_cta * upr << (p.log_tokens + 1)) <= 5 * kThreads &&
           p.num_tokens >> (p.log_tokens + 1) >= 152 && kThreads >> (p.log_tokens + 1) >= upr)
        ++p.log_tokens;
    const dim3 grid((p.num_tokens + (1 << p.log_tokens) - 1) >> p.log_tokens,
                    (p.num_heads + p.heads_per_cta - 1) / p.heads_per_cta);
    p.prefetch = static_cast<int64_t>(p.num_tokens) * p.num_heads * p.head_dim >= 1 << 19;
    const size_t smem = sizeof(float) * (rope.rotary_dim << p.log_tokens);
    return wide ? launch_pdl(rotary_kernel<8, AXES>, grid, dim3(kThreads), smem, stream, rope, p)
                : launch_pdl(rotary_kernel<4, AXES>, grid, dim3(kThreads), smem, stream, rope, p);
}

template <bool AXES>
cudaError_t launch_append_t(int head_dim, int kind, const RopeArg<AXES> &rope, const AppendParams &p0, cudaStream_t stream) {
    AppendParams p = p0;
    if (p.num_tokens <= 0 || p.num_reqs <= 0) return cudaSuccess;
    p.q_heads_per_cta = p.num_heads_q < 32 ? p.num_heads_q : 32;
    const int q_parts = p.q == nullptr ? 0 : (p.num_heads_q + p.q_heads_per_cta - 1) / p.q_heads_per_cta;
    const dim3 grid(p.num_tokens / kBlockSize + 2 * p.num_reqs, 2 * ((p.num_heads_kv + 7) / 8) + q_parts);
    const bool wide = wide_units(rope, head_dim);
    if (head_dim == 128)
        return wide ? launch_append_d<128, 8, AXES>(kind, rope, p, grid, stream)
                    : launch_append_d<128, 4, AXES>(kind, rope, p, grid, stream);
    if (head_dim == 64)
        return wide ? launch_append_d<64, 8, AXES>(kind, rope, p, grid, stream)
                    : launch_append_d<64, 4, AXES>(kind, rope, p, grid, stream);
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_rotary(const RopeParams &rope, const RotaryParams &p, cudaStream_t stream) {
    return launch_rotary_t<false>(rope, p, stream);
}

cudaError_t launch_rotary_axes(const AxesRopeParams &rope, const RotaryParams &p, cudaStream_t stream) {
    return launch_rotary_t<true>(rope, p, stream);
}

cudaError_t launch_append(int head_dim, int kind, const RopeParams &rope, const AppendParams &p, cudaStream_t stream) {
    return launch_append_t<false>(head_dim, kind, rope, p, stream);
}

cudaError_t launch_append_axes(int head_dim, int kind, const AxesRopeParams &rope, const AppendParams &p, cudaStream_t stream) {
    return launch_append_t<true>(head_dim, kind, rope, p, stream);
}

}  // namespace pa
