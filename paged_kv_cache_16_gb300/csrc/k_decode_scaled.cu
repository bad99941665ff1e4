// Split-KV decode attention over block-scaled 8-bit caches: E4M3 or int8
// codes with one scale per (cache block, kv head) for K and for V.
//
// For one query row with scores s_j = c <q, kcode_j> ks_b(j) (c =
// softmax_scale * log2 e, b(j) the block of key j) and values vcode_j vs_b(j):
//   w_j = 2^(s_j + log2 vs_b(j) - R),  R >= max_j (s_j + log2 vs_b(j)) - 8
//   O = sum_j w_j vcode_j,   L = sum_j w_j / vs_b(j),   out = O / L.
// The value scales go into the exponents, so the codes feed the tensor cores
// unscaled, and the reference R bounds the weights as the products see them:
// whatever the scales of other blocks, the largest term of O keeps the f16
// weights' full precision (weights <= 2^8, R moves when it grows by more than
// 2^8), and a weight lost to f16's underflow is below 2^-24 of it.  L is summed
// in fp32, per block, times 1 / vs.
//
// GB300 mapping: persistent CTAs over equal cuts of the concatenated key blocks,
// a producer warp that streams each block as one TMA box for K and one for V
// (all HG kv heads of the CTA) into an mbarrier ring, one consumer warp per kv
// head, partials joined by the merge kernel.  The scales of a block (4 bytes per
// head and tensor, one sector for 8 heads) are copied into the stage by the
// producer's lanes with 4-byte cp.async that arrive on the stage's barrier: no
// lane waits for them.  Products are computed transposed (S^T = K Q^T, O^T +=
// V^T P^T): the 16 keys of a block are the MMA rows, the query rows (token,
// head) its columns, NT tiles of 8 of them, so a code is converted to f16 once
// for all query rows.
//
// Bound by HBM: 8 contexts of 131072 int8 keys (Hq 64, Hkv 8, D 128) 319 us with
// the merge, 6.7 TB/s (0.99 of the copy rate; 312 without the copies of the
// scales); 64 contexts of 540..4068 53 us, 5.7 TB/s around the ring's fill, the tail
// and the merge (51 with the consumers' arithmetic taken out); 128 rows of 4
// tokens over E4M3 206 us (196).
#include <type_traits>

#include "dev.cuh"

namespace pa {
namespace {

using namespace dev;

template <int D, int HG>
struct ScaledCfg {
    static constexpr int BOX = kBlockSize * D;             // one head's [16 rows][D] codes
    static constexpr int TSTAGE = HG * BOX;                // K (or V) codes of a block
    static constexpr int STAGE = decode_stage_bytes(D, HG, true);
    static constexpr int NS = decode_stages(D, HG, true);
    static constexpr int THREADS = decode_threads(HG);
    static constexpr int SMEM = scaled_decode_smem_bytes(D, HG);
    static_assert(STAGE == 2 * TSTAGE);
};

// Byte offset of the 16-byte chunk `chunk` of row `row` in a head's tile, as TMA
// lays it out: rows of 128 bytes with 128-byte swizzling (chunk ^= row mod 8) or
// of 64 bytes with 64-byte swizzling (chunk ^= row / 2 mod 4).
template <int D>
__device__ __forceinline__ uint32_t tile_at(uint32_t row, uint32_t chunk) {
    if constexpr (D == 128) return row * 128u + ((chunk ^ (row & 7u)) << 4);
    else return row * 64u + ((chunk ^ ((row >> 1) & 3u)) << 4);
}

__device__ __forceinline__ float lds_f32(uint32_t addr) { return __uint_as_float(lds_u32(addr)); }

__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
// arrive on `bar` (one of its counted arrivals) once this thread's earlier
// cp.async copies have landed
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// Words of a lane's piece of one value row: D / 8 codes.
template <int D>
struct Piece {
    uint32_t w[D / 32];
    __device__ __forceinline__ void load(uint32_t vb, uint32_t row, uint32_t g) {
        if constexpr (D == 128) {
            const uint4 v = lds_v4(vb + tile_at<D>(row, g));
            w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
        } else {
            const uint2 v = lds_v2(vb + tile_at<D>(row, g >> 1) + 8u * (g & 1u));
            w[0] = v.x; w[1] = v.y;
        }
    }
};

// WIN: with a sliding window and first tokens (items in WindowView's numbers).
template <int D, int HG, bool INT8, bool WIN>
struct Consumer {
    using C = ScaledCfg<D, HG>;
    static constexpr int CH = D / 64;   // 16-byte chunks of a key row per lane of a quad
    static constexpr float kUnset = -1e30f;
    const ScaledDecodeParams &p;
    uint32_t stage0, scale0, full0, empty0;   // shared memory: stages, scales, barriers
    volatile int *abort_flag;
    int warp, lane, g, t4;
    int slot = 0;         // next stage of the ring and the parity of its phase
    uint32_t parity = 0;

    // One item, NT tiles of 8 query rows.  The contraction runs over a permuted
    // order of dims: step (h, w) takes, from lane t of a quad, the four dims
    // 16 (CH t + h) + 4 w .. + 3, so a lane reads its keys' codes (and q) in
    // 16-byte chunks.  Lane (g, t) holds, of tile n, the scores of keys g and
    // g + 8 for the rows 8n + 2t and 8n + 2t + 1; of a value row it reads the
    // dims of its piece, D / 8 from D / 8 g on, and of O the same dims for the
    // two rows: dim 4j + {0, 1, 2, 3} of the piece of row e in
    // ot[n][2j][e], ot[n][2j][2 + e], ot[n][2j + 1][e], ot[n][2j + 1][2 + e].
    template <int NT>
    __device__ __forceinline__ bool run(const DecodeItem &item) {
        const DecodeParams &b = p.base;
        const int G = b.group;
        const int kvh = item.head_group * HG + warp;
        const int nrow = item.n_tok * G;
        // q as f16, each row scaled by a power of two to magnitudes below 2 (4 for
        // the largest of bf16, whose range does not fit f16's): the factor returns
        // in the scores.  Exact for elements down to 2^-17 of the row's largest
        // magnitude; smaller ones are rounded to steps of 2^-24 of it, at most
        // 2^-25 of it off (a score by 2^-25 of that magnitude times the sum of |k|).
        // f16 and not bf16, because one conversion then serves the codes of K and V
        uint32_t qt[NT][D / 16][2];
        float rf[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int r = 8 * n + g;
            const uint16_t *qg = b.q + (static_cast<int64_t>(item.token + r / G) * b.num_heads_q + kvh * G + r % G) * D;
            float amax = 0.f;
#pragma unroll
            for (int h = 0; h < CH; ++h)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    uint4 v = make_uint4(0, 0, 0, 0);
                    if (r < nrow) v = __ldg(reinterpret_cast<const uint4 *>(qg + 16 * (CH * t4 + h)) + i);
                    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        qt[n][4 * h + 2 * i + k / 2][k & 1] = w[k];
                        amax = max3(amax, fabsf(bf16_lo(w[k])), fabsf(bf16_hi(w[k])));
                    }
                }
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
            const int e2 = min(max(static_cast<int>(__float_as_uint(amax) >> 23) - 127, -126), 126);
            const float down = __uint_as_float(static_cast<uint32_t>(127 - e2) << 23);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    qt[n][kk][e] = pack_f16x2(bf16_lo(qt[n][kk][e]) * down, bf16_hi(qt[n][kk][e]) * down);
            const float up = __uint_as_float(static_cast<uint32_t>(127 + e2) << 23) * b.scale_log2;
#pragma unroll
            for (int e = 0; e < 2; ++e) rf[n][e] = __shfl_sync(0xffffffffu, up, 4 * (2 * t4 + e));   // of row 8n + 2t + e
        }
        const int lim_lo = item.key_end - (item.n_tok - 1);
        // windows begin below low_top, the item's first one at low_min
        const int low_top = item.key_end - b.window, low_min = lim_lo - b.window;
        float ot[NT][D / 16][4], lt[NT][2], ref[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int j = 0; j < D / 16; ++j) ot[n][j][0] = ot[n][j][1] = ot[n][j][2] = ot[n][j][3] = 0.f;
            lt[n][0] = lt[n][1] = 0.f;
            ref[n][0] = ref[n][1] = kUnset;
        }

        auto qk = [&](uint32_t kb, float (&s)[NT][4]) {
#pragma unroll
            for (int h = 0; h < CH; ++h) {
                const uint4 k0 = lds_v4(kb + tile_at<D>(g, CH * t4 + h)), k1 = lds_v4(kb + tile_at<D>(g + 8, CH * t4 + h));
                const uint32_t w0[4] = {k0.x, k0.y, k0.z, k0.w}, w1[4] = {k1.x, k1.y, k1.z, k1.w};
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    uint32_t a[4];
                    codes_to_f16<INT8>(w0[w], a[0], a[2]);
                    codes_to_f16<INT8>(w1[w], a[1], a[3]);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        if (h == 0 && w == 0) mma_f16_16816_first(s[n], a, qt[n][0][0], qt[n][0][1]);
                        else mma_f16_16816(s[n], a, qt[n][4 * h + w][0], qt[n][4 * h + w][1]);
                    }
                }
            }
        };
        // O^T += V^T P^T of one block; codes of rows that are not `live` (MASKED:
        // they may be anything, also NaN) count as 0
        auto pv = [&](auto masked, uint32_t vb, const uint32_t (&w)[NT][2], const LiveRows<WIN> &live) {
            Piece<D> v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = 2 * t4 + (i & 1) + 8 * (i >> 1);
                v[i].load(vb, row, g);
                if constexpr (decltype(masked)::value) {
#pragma unroll
                    for (int j = 0; j < D / 32; ++j) v[i].w[j] = live.has(row) ? v[i].w[j] : 0u;
                }
            }
#pragma unroll
            for (int j = 0; j < D / 32; ++j) {
                uint32_t a0[4], a1[4];
                codes_to_f16<INT8>(prmt(v[0].w[j], v[1].w[j], 0x5140u), a0[0], a0[1]);
                codes_to_f16<INT8>(prmt(v[2].w[j], v[3].w[j], 0x5140u), a0[2], a0[3]);
                codes_to_f16<INT8>(prmt(v[0].w[j], v[1].w[j], 0x7362u), a1[0], a1[1]);
                codes_to_f16<INT8>(prmt(v[2].w[j], v[3].w[j], 0x7362u), a1[2], a1[3]);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    mma_f16_16816(ot[n][2 * j], a0, w[n][0], w[n][1]);
                    mma_f16_16816(ot[n][2 * j + 1], a1, w[n][0], w[n][1]);
                }
            }
        };
        // one softmax round over one (TWO = false) or two blocks
        auto round = [&](auto two_c, int pg) -> bool {
            constexpr int NB = decltype(two_c)::value ? 2 : 1;
            uint32_t st[NB], fin[NB];
            float sc[NB][NT][4], kf[NB][NT][2], lv[NB];
#pragma unroll
            for (int k = 0; k < NB; ++k) {
                if (!warp_wait(full0 + 8u * slot, parity, abort_flag)) return false;
                st[k] = stage0 + static_cast<uint32_t>(slot) * C::STAGE + warp * C::BOX;
                fin[k] = empty0 + 8u * slot;
                const uint32_t sa = scale0 + 4u * (2 * HG * slot + warp);
                // (a NaN value scale shows in the scores, where masks can take it out)
                const float vs = used_scale(lds_f32(sa + 4u * HG));
                const float ks = vs == vs ? used_scale(lds_f32(sa)) : vs;
                lv[k] = vs == vs ? lg2(vs) : 0.f;
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) kf[k][n][e] = score_factor(ks, rf[n][e]);
                if (++slot == C::NS) {
                    slot = 0;
                    parity ^= 1u;
                }
            }
#pragma unroll
            for (int k = 0; k < NB; ++k) qk(st[k], sc[k]);
            const int key0 = pg * kBlockSize;
            if (lim_lo - key0 < NB * kBlockSize) {
                // token i of the item sees keys < key_end - (n_tok - 1 - i)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int lim = min(item.key_end, lim_lo + (8 * n + 2 * t4 + e) / G) - key0;
#pragma unroll
                        for (int k = 0; k < NB; ++k) {
                            if (16 * k + g >= lim) sc[k][n][e] = -INFINITY;
                            if (16 * k + g + 8 >= lim) sc[k][n][e + 2] = -INFINITY;
                            if (16 * k >= lim) kf[k][n][e] = 1.f;   // none of the block: its scale, NaN even, plays no part
                        }
                    }
            }
            if (WIN && key0 < low_top) {
                // keys behind a row's window that are not first tokens
                const int first = b.sinks - key0;
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int low = min(item.key_end, lim_lo + (8 * n + 2 * t4 + e) / G) - b.window - key0;
                        auto behind = [&](int i) { return i >= first && i < low; };
#pragma unroll
                        for (int k = 0; k < NB; ++k) {
                            if (behind(16 * k + g)) sc[k][n][e] = -INFINITY;
                            if (behind(16 * k + g + 8)) sc[k][n][e + 2] = -INFINITY;
                            if (behind(16 * k) && behind(16 * k + 15)) kf[k][n][e] = 1.f;   // none of the block
                        }
                    }
            }
            bool grow = false;
            float mx[NT][2];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float m = fmaf(fmaxf(sc[0][n][e], sc[0][n][e + 2]), kf[0][n][e], lv[0]);
                    if constexpr (NB == 2) m = fmaxf(m, fmaf(fmaxf(sc[1][n][e], sc[1][n][e + 2]), kf[1][n][e], lv[1]));
                    mx[n][e] = m;
                }
#pragma unroll
            for (int o = 4; o < 32; o <<= 1)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) mx[n][e] = fmaxf(mx[n][e], __shfl_xor_sync(0xffffffffu, mx[n][e], o));
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) grow |= mx[n][e] > ref[n][e] + 8.f;
            if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float a[2] = {1.f, 1.f};
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        if (mx[n][e] > ref[n][e] + 8.f) {
                            a[e] = ex2(ref[n][e] - mx[n][e]);
                            ref[n][e] = mx[n][e];
                            lt[n][e] *= a[e];
                        }
#pragma unroll
                    for (int j = 0; j < D / 16; ++j) {
                        ot[n][j][0] *= a[0]; ot[n][j][1] *= a[1]; ot[n][j][2] *= a[0]; ot[n][j][3] *= a[1];
                    }
                }
            }
            uint32_t w[NB][NT][2];
#pragma unroll
            for (int k = 0; k < NB; ++k) {
                const float iv = ex2(-lv[k]);   // 1 / vs, the inverse of what the exponents hold
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float x[4];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float c = lv[k] - ref[n][e];
                        x[e] = ex2(fmaf(sc[k][n][e], kf[k][n][e], c));
                        x[e + 2] = ex2(fmaf(sc[k][n][e + 2], kf[k][n][e], c));
                        lt[n][e] = fmaf(x[e] + x[e + 2], iv, lt[n][e]);
                    }
                    // P^T as B fragments: rows (8n + 2t, 8n + 2t + 1) of key g
                    // (g + 8), transposed 8x8
                    w[k][n][0] = movmatrix_trans(pack_f16x2(x[0], x[1]));
                    w[k][n][1] = movmatrix_trans(pack_f16x2(x[2], x[3]));
                }
            }
#pragma unroll
            for (int k = 0; k < NB; ++k) {
                const LiveRows<WIN> live(key0 + k * kBlockSize, item.key_end, b.sinks, low_min);
                if (!live.all()) pv(std::true_type{}, st[k] + C::TSTAGE, w[k], live);
                else pv(std::false_type{}, st[k] + C::TSTAGE, w[k], live);
            }
            __syncwarp();
            if (lane == 0) {
#pragma unroll
                for (int k = 0; k < NB; ++k) mbar_arrive(fin[k]);
            }
            return true;
        };
        int pg = item.page_begin;
        for (; pg + 1 < item.page_end; pg += 2)
            if (!round(std::true_type{}, pg)) return false;
        if (pg < item.page_end && !round(std::false_type{}, pg)) return false;

        // ------------------------------------------------------ finalize --
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float l = lt[n][e];
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
                const int r = 8 * n + 2 * t4 + e;
                if (r >= nrow) continue;
                // a NaN stays one; no visible key: 0
                const float inv = l == 0.f ? 0.f : 1.f / l;
                const int tok = item.token + r / G, head = kvh * G + r % G;
                auto o4 = [&](int j) {   // dims 4j .. 4j + 3 of the piece
                    return make_float4(ot[n][2 * j][e] * inv, ot[n][2 * j][2 + e] * inv, ot[n][2 * j + 1][e] * inv,
                                       ot[n][2 * j + 1][2 + e] * inv);
                };
                if (item.part < 0) {
                    uint16_t *o = b.out + (static_cast<int64_t>(tok) * b.num_heads_q + head) * D + D / 8 * g;
#pragma unroll
                    for (int j = 0; j < D / 32; j += 2) {
                        const float4 x = o4(j), y = o4(j + 1);
                        *reinterpret_cast<uint4 *>(o + 4 * j) = make_uint4(pack_bf16x2(x.x, x.y), pack_bf16x2(x.z, x.w),
                                                                           pack_bf16x2(y.x, y.y), pack_bf16x2(y.z, y.w));
                    }
                } else {
                    const int64_t slot_at = static_cast<int64_t>(b.part_offset[tok * b.n_groups + item.head_group]) + item.part;
                    float *o = b.o_part + (slot_at * b.num_heads_q + head) * D + D / 8 * g;
#pragma unroll
                    for (int j = 0; j < D / 32; ++j) *reinterpret_cast<float4 *>(o + 4 * j) = o4(j);
                    // the partial's weight in the merge is 2^m l: kept as l = 1, so
                    // that L's own range (1 / vs) does not enter there; a NaN
                    // takes the merge over
                    if (g == 0)
                        b.ml_part[slot_at * b.num_heads_q + head] =
                            l == 0.f ? make_float2(-INFINITY, 0.f)
                                     : make_float2(l != l ? 3.0e38f : ref[n][e] + lg2(l), 1.f);
                }
            }
        return true;
    }
};

template <int D, int HG, bool INT8, bool WIN>
__global__ void __launch_bounds__((HG + 1) * 32, scaled_decode_ctas_per_sm(D, HG))
scaled_decode_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                     const ScaledDecodeParams sp) {
    using C = ScaledCfg<D, HG>;
    const DecodeParams &p = sp.base;
    extern __shared__ uint8_t smem_raw[];
    __shared__ int abort_flag;
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;      // stages, 1024-aligned
    const uint32_t bar0 = base + C::NS * C::STAGE;                    // full | empty | scales
    auto full = [&](int s) { return bar0 + 8u * s; };
    auto empty = [&](int s) { return bar0 + 8u * (C::NS + s); };
    const uint32_t scale0 = bar0 + 16u * C::NS;                       // [stage][K, V][head] floats
    auto stage = [&](int s) { return base + static_cast<uint32_t>(s) * C::STAGE; };

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    grid_launch_dependents();
    if (threadIdx.x == 0) {
        abort_flag = 0;
        for (int s = 0; s < C::NS; ++s) {
            mbar_init(full(s), 33);      // the codes' byte count, and one arrival per producer lane for the scales
            mbar_init(empty(s), HG);
        }
        fence_barrier_init();
    } else if (threadIdx.x == 32 * HG) {
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
    }
    // everything below reads or writes what earlier kernels of the stream
    // produce or consume (work list, caches, partials)
    grid_dep_wait();
    __syncthreads();

    const int item_begin = p.cta_begin[blockIdx.x];
    const int item_end = p.cta_begin[blockIdx.x + 1];

    if (warp == HG) {
        // ------------------------------------------------------ producer --
        int issued = 0;
        const uint64_t evict_first = policy_evict_first();   // the stream is read once
        bool ok = true;
        // lane l < 2 HG copies the scale of tensor l / HG, head l % HG
        const float *scales = lane / HG == 0 ? sp.key_scales : sp.value_scales;
        for (int it = item_begin; it < item_end && ok; ++it) {
            DecodeItem item = p.items[it];
            const WindowView view = own_numbers<WIN>(p, item);
            const int32_t *bt = p.block_table + static_cast<int64_t>(item.req) * p.max_blocks;
            const int h0 = item.head_group * HG;
            int32_t blk_lane = 0;       // block id of page (window + lane), 32 pages at a time
            int window = item.page_begin - 32;
            for (int pg = item.page_begin; pg < item.page_end; ++pg) {
                if (pg - window >= 32) {
                    window = pg;
                    blk_lane = pg + lane < item.page_end ? bt[WIN ? min(view.at(pg + lane), p.max_blocks - 1) : pg + lane] : 0;
                }
                const int s = issued % C::NS;
                const int n = issued / C::NS;
                if (n > 0 && !warp_wait(empty(s), (n & 1) ^ 1, &abort_flag)) {
                    if (lane == 0) raise_abort(&abort_flag, p.err, kErrTimeout);
                    ok = false;
                    break;
                }
                const int32_t blk = __shfl_sync(0xffffffffu, blk_lane, pg - window);
                const bool valid = blk >= 0 && blk < p.num_blocks;
                if (lane == 0) {
                    if (valid) {
                        mbar_arrive_expect_tx(full(s), C::STAGE);
                    } else {
                        atomicOr(p.err, kErrBlockRange);
                        mbar_arrive(full(s));
                    }
                }
                __syncwarp();
                if (valid) {
                    if (lane < 2)
                        tma_load_3d_hint(stage(s) + lane * C::TSTAGE, lane ? &tm_v : &tm_k, 0, blk * kBlockSize, h0, full(s),
                                         evict_first);
                    if (lane < 2 * HG)
                        cp_async4(scale0 + 4u * (2 * HG * s + lane),
                                  scales + static_cast<int64_t>(blk) * p.num_heads_kv + h0 + lane % HG);
                }
                cp_async_arrive(full(s));
                ++issued;
            }
        }
        // Never leave the CTA with copies in flight.
        if (lane == 0) {
            for (int k = issued - 1; k >= 0 && k >= issued - C::NS; --k)
                if (!mbar_wait(full(k % C::NS), (k / C::NS) & 1, nullptr)) atomicOr(p.err, kErrTimeout);
        }
    } else {
        // ----------------------------------------------------- consumers --
        Consumer<D, HG, INT8, WIN> c{sp, base, scale0, bar0, bar0 + 8u * C::NS, &abort_flag, warp, lane, lane >> 2, lane & 3};
        bool ok = true;
        for (int it = item_begin; it < item_end && ok; ++it) {
            DecodeItem item = p.items[it];
            own_numbers<WIN>(p, item);
            ok = item.n_tok * p.group <= 8 ? c.template run<1>(item) : c.template run<2>(item);
            if (!ok && lane == 0) raise_abort(&abort_flag, p.err, kErrTimeout);
        }
    }
    __syncthreads();
}

template <int D, int HG, bool INT8, bool WIN>
cudaError_t configure() {
    // the attribute is per function and device; setting it again is harmless
    return cudaFuncSetAttribute(scaled_decode_kernel<D, HG, INT8, WIN>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                ScaledCfg<D, HG>::SMEM);
}

template <int D, int HG, bool INT8, bool WIN>
cudaError_t launch_t(int num_ctas, const CUtensorMap &tm_k, const CUtensorMap &tm_v, const ScaledDecodeParams &p,
                     cudaStream_t stream) {
    using C = ScaledCfg<D, HG>;
    return launch_pdl(scaled_decode_kernel<D, HG, INT8, WIN>, dim3(num_ctas), dim3(C::THREADS), C::SMEM, stream, tm_k, tm_v, p);
}

}  // namespace

#define PA_SCALED_CASES(X)                                                                                       \
    X(64, 1, false) X(64, 2, false) X(64, 4, false) X(64, 8, false) X(128, 1, false) X(128, 2, false)           \
    X(128, 4, false) X(128, 8, false) X(64, 1, true) X(64, 2, true) X(64, 4, true) X(64, 8, true) X(128, 1, true) \
    X(128, 2, true) X(128, 4, true) X(128, 8, true)

cudaError_t prepare_scaled_decode(int head_dim, int hg, bool int8, bool window) {
#define X(d, h, i) \
    if (head_dim == d && hg == h && int8 == i) return window ? configure<d, h, i, true>() : configure<d, h, i, false>();
    PA_SCALED_CASES(X)
#undef X
    return cudaErrorInvalidValue;
}

cudaError_t launch_scaled_decode(int head_dim, int hg, bool int8, int num_ctas, const CUtensorMap &tm_k,
                                 const CUtensorMap &tm_v, const ScaledDecodeParams &p, cudaStream_t stream) {
    if (num_ctas <= 0) return cudaSuccess;
#define X(d, h, i) \
    if (head_dim == d && hg == h && int8 == i)  \
        return p.base.window > 0 ? launch_t<d, h, i, true>(num_ctas, tm_k, tm_v, p, stream) \
                                 : launch_t<d, h, i, false>(num_ctas, tm_k, tm_v, p, stream);
    PA_SCALED_CASES(X)
#undef X
    return cudaErrorInvalidValue;
}

}  // namespace pa
