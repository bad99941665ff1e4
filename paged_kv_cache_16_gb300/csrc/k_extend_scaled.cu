// Extend / chunked-prefill and shared-prefix attention on the tensor cores over
// block-scaled 8-bit caches: the schedule of k_extend.cu (two 128-row sub-tiles
// per CTA tile against shared 128-key tiles; TMA producer, one MMA-issuing thread,
// a softmax warpgroup per sub-tile, accumulators in tensor memory), with the codes
// themselves as operands.  K and V tiles are 16-bit copies of the codes, exact: K
// in bf16 beside the bf16 queries, V in f16 beside f16 weights.  The scales enter
// in fp32, per block of 16 key columns, as in the split-KV kernel:
//   w = 2^(s + log2 vs - R), s = softmax_scale log2(e) ks <q, kcode>,
//   O += w vcode,  L += (sum of the block's w) / vs,  out = O / L,
// so a tile loses nothing to the quantisation's form (bf16 weights and dequantised
// bf16 K and V gave 2.6 times the error of the output's own rounding; this adds
// nothing visible).  Three factors per (block, kv head), written by the expansion
// kernel as one 16-byte record, travel with the V stage, which is not given back
// before its weights have been used: a softmax warp waits for it under QK^T.
//
// Two chunks of 2048 tokens over 2304 and 4864 (Hq 32, Hkv 8, D 128): 200 us at
// 2070 MHz, 1546 TFLOP/s, where the kernel of the E4M3 caches with one scale takes
// 192 on the same schedule (no factors; bf16 weights).  A step of 128 keys has 2048 cycles of MMAs and takes ~2800 (tensor pipe
// active 68%, issue 43%): what the MMA warp does between two MMAs, and the chain
// S -> softmax -> P of a sub-tile (~1500 cycles), which its own PV and QK^T follow.
// P is handed over in halves, so that PV begins under the second half's
// exponentials (3%; after a quarter or three quarters 1% more than that), by one
// arrival per warp (1.5%).  Between two tiles go ~3 steps' time: the last softmax,
// the epilogue and the first QK^T in a row.  Measured and not kept, as parts of the
// time then: ring indices by division and all commits at the groups' ends +8%;
// weights through shared memory, QK^T a step ahead, +23% (every operand from shared
// memory fills its bandwidth); one S buffer for both sub-tiles and QK^T a step
// ahead, +39% with one MMA thread, +11% with one for QK^T and one for PV; an MMA
// thread per sub-tile, +25%, taking turns at the pipe +2%; two threads per row +15%;
// the first half's weights against the old reference, checked by their sum, beside
// the second half's maximum, S read again where a row needs a new one, +3%; the
// blocks' factors read from shared memory where they are used instead of held, +2%;
// the next tile's first QK^T in a tile's last step +2%, one loop body for full and
// last steps +23%; stages given back by a softmax warp, tile descriptions in shared
// memory, three K and two V stages: no change.
//
// 4096 tokens over 12288, a window of 4096 with 64 first tokens: 210 us beside the
// 8 of the expansion (tensor pipe 55% active): 456 whole tiles of 34 steps in three
// rounds, the last 56 halved; all 512 whole in four rounds 247 with the expansion, the
// last ones' keys cut in two and merged 234.
#include "tiles.cuh"

namespace pa {
namespace {

using namespace dev;
using namespace tiles;

template <int D>
struct ScaledExtCfg {
    static constexpr int NH = D / 64;
    static constexpr int HALF = 128 * 128;            // [128 rows][64] bf16 half tile
    static constexpr int QB = NH * HALF;              // one Q sub-tile
    static constexpr int KVB = NH * HALF;             // K (or V) tile bytes per stage
    static constexpr int NSK = 2;                     // K stages
    static constexpr int NSV = 3;                     // V stages (V waits longest for its stage)
    static constexpr int THREADS = 384;               // 3 warpgroups
    // registers per thread after the split (launch: 168 x 384 = 64512):
    // 120 x 128 for the load / MMA warpgroup + 192 x 256 for the two softmax
    // warpgroups = 64512
    static constexpr int REGS_CTRL = 120;
    static constexpr int REGS_SOFTMAX = 192;
    static_assert(REGS_CTRL * 128 + REGS_SOFTMAX * 256 <= 168 * 384, "register split exceeds the launch");
    static constexpr int FACTORS = NSV * (kTileKeys / kBlockSize) * 16;   // a record per block of a V stage
    static constexpr int TILE_SMEM = 2 * QB + (NSK + NSV) * KVB + FACTORS;
    // one CTA per SM: it owns all 512 tensor-memory columns
    static constexpr int SMEM = (TILE_SMEM + 1024 < 120 * 1024) ? 120 * 1024 : TILE_SMEM + 1024;
    static constexpr uint32_t TMEM_COLS = 512;
    static constexpr uint32_t IDESC_QK = idesc_bf16(128, 128, false, false);
    static constexpr uint32_t IDESC_PV = idesc_bf16(128, D, false, true) & ~((1u << 7) | (1u << 10));   // f16 A and B
};


// WIN: with a sliding window and first tokens (tiles in WindowView's numbers, the
// head padded to whole key tiles: the copies of a head's blocks are consecutive,
// and so are those from the window on).  SPLIT: tiles of one sub-tile of rows whose
// keys both sub-tiles share may be among them.
template <int D, bool WIN, bool SPLIT>
__global__ void __launch_bounds__(384, 1)
scaled_extend_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
              const __grid_constant__ CUtensorMap tm_v, const ScaledExtendParams sp) {
    using C = ScaledExtCfg<D>;
    const ExtendParams &p = sp.base;
    extern __shared__ uint8_t smem_raw[];
    __shared__ int abort_flag;
    __shared__ uint32_t tmem_base_slot;
    __shared__ __align__(8) uint64_t bars[NUM_BARS];
    __shared__ float2 second[SPLIT ? kTileRows : 1];   // split tiles: sub-tile 1's maximum and sum of each row

    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    auto q_s = [&](int t) { return base + static_cast<uint32_t>(t) * C::QB; };
    auto k_s = [&](int s) { return base + 2 * C::QB + static_cast<uint32_t>(s) * C::KVB; };
    auto v_s = [&](int s) { return base + 2 * C::QB + static_cast<uint32_t>(C::NSK + s) * C::KVB; };
    // factors of block `page` of V stage s: {ks * scale, log2 vs, 1 / vs, unused}
    auto f_s = [&](int s, int page) {
        return base + 2 * C::QB + static_cast<uint32_t>(C::NSK + C::NSV) * C::KVB + 16u * (8 * s + page);
    };
    auto bar = [&](int i) { return smem_u32(&bars[i]); };

    grid_launch_dependents();
    grid_dep_wait();    // the work list and caches come from earlier kernels of the stream
    // this CTA's tiles, longest first (the planner's greedy assignment)
    const int tile_begin = p.cta_tile_begin[blockIdx.x];
    const int tile_end = p.cta_tile_begin[blockIdx.x + 1];
    if (tile_begin >= tile_end) return;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);   // (uniform to the compiler)
    const int lane = threadIdx.x & 31;
    const int G = p.group;
    const int tpt = kTileRows / G;                    // tokens per 128-row sub-tile

    if (threadIdx.x == 0) {
        abort_flag = 0;
        mbar_init(bar(B_QFULL), 1);
        mbar_init(bar(B_QEMPTY), 1);
        for (int s = 0; s < C::NSK; ++s) {
            mbar_init(bar(B_KFULL + s), 1);
            mbar_init(bar(B_KEMPTY + s), 1);
        }
        for (int s = 0; s < C::NSV; ++s) {
            mbar_init(bar(B_VFULL + s), 1);
            mbar_init(bar(B_VEMPTY + s), 1);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(bar(B_SFULL + t), 1);
            mbar_init(bar(B_PFULL + t), 4);       // a warp each
            mbar_init(bar(B_PFULL + 2 + t), 4);
            mbar_init(bar(B_ODONE + t), 1);
        }
        mbar_init(bar(B_DRAIN), 1);
        mbar_init(bar(B_SECOND), 4);
        mbar_init(bar(B_JOINED), 4);
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(&tmem_base_slot), C::TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_base_slot;
    if (warp < 4) {
      // warpgroup 0: loads and MMA issue, with few registers
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::REGS_CTRL));
      if (warp == 0) {
        // -------------------------------------------------------- producer --
        if (lane == 0) {
            tma_prefetch_desc(&tm_q);
            tma_prefetch_desc(&tm_k);
            tma_prefetch_desc(&tm_v);
        }
        int issued[2] = {0, 0};   // K and V tiles whose loads were issued (over all tiles)
        int n_q_loads = 0;
        bool ok = true;
        for (int ti = tile_begin; ti < tile_end && ok; ++ti) {
            const ExtendTile tile = p.tiles[p.cta_tiles[ti]];
            const TileShape sh = tile_shape<SPLIT>(tile, tpt);
            // Q of this tile, once the previous tile's QK^T no longer read Q
            if (n_q_loads > 0 && !warp_wait(bar(B_QEMPTY), (n_q_loads - 1) & 1, &abort_flag)) {
                if (lane == 0) raise_abort(&abort_flag, p.err, kErrTimeout);
                break;
            }
            const int n_q = sh.n_sub[1] > 0 ? 2 : 1;
            // each box is tpt tokens x G heads x 64 dims: tpt * G rows of
            // 128 bytes (128 rows unless G does not divide 128)
            if (lane == 0) mbar_arrive_expect_tx(bar(B_QFULL), n_q * C::NH * tpt * G * 128);
            __syncwarp();
            if (lane < n_q * C::NH) {
                const int t = lane / C::NH, half = lane % C::NH;
                tma_load_3d(q_s(t) + half * C::HALF, &tm_q, half * 64, tile.kv_head * G,
                            tile.t0 + (sh.split ? 0 : t * tpt), bar(B_QFULL));
            }
            ++n_q_loads;
            // the copies of a request's blocks are consecutive, so a key tile is
            // 128 consecutive rows of them: one box per 64 columns of K and of V
            // (16 boxes of one block each and 8 bulk copies of single records cost
            // the producer 8% of the kernel's time).  Rows behind the key range
            // belong to other requests or to none: masked columns, and value
            // rows that the softmax warps zero
            const int32_t *copies = p.block_table + static_cast<int64_t>(tile.req) * p.max_blocks;
            const int pg_begin = tile.key_begin / kBlockSize;
            const int pg_end = (tile.key_end - tile.key_begin + kBlockSize - 1) / kBlockSize;
            // windowed: first the copies of the head (rows of its padding are other
            // blocks'), then those from page `head` on; all counted from the tile's
            // first page
            const int head = WIN ? tile.head - pg_begin : 0, head_end = head_blocks(p.sinks, p.sinks) - pg_begin;
            const int32_t dst0 = WIN ? copies[tile.head + tile.skip] - head : copies[pg_begin];
            const int32_t head0 = head > 0 ? copies[0] + pg_begin : 0;
            if (dst0 + max(head, 0) < 0 || dst0 + pg_end > p.num_blocks ||
                head0 < 0 || (head > 0 && head0 + min(head_end, pg_end) > p.num_blocks)) {   // (not from the planner)
                if (lane == 0) raise_abort(&abort_flag, p.err, kErrBlockRange);
                break;
            }
            for (int j = 0; j < sh.n_tiles; ++j) {
                const int pg0 = j * (kTileKeys / kBlockSize);
                const bool in_head = pg0 < head;
                const int pages = min(kTileKeys / kBlockSize, (in_head ? min(head_end, pg_end) : pg_end) - pg0);
                const int32_t at = (in_head ? head0 : dst0) + pg0;
#pragma unroll
                for (int tensor = 0; tensor < 2; ++tensor) {
                    const int ns = tensor ? C::NSV : C::NSK;
                    const int s = issued[tensor] % ns, n = issued[tensor] / ns;
                    const int empty = tensor ? B_VEMPTY : B_KEMPTY;
                    const int full = tensor ? B_VFULL : B_KFULL;
                    if (n > 0 && !warp_wait(bar(empty + s), (n & 1) ^ 1, &abort_flag)) {
                        if (lane == 0) raise_abort(&abort_flag, p.err, kErrTimeout);
                        ok = false;
                        break;
                    }
                    if (lane == 0) mbar_arrive_expect_tx(bar(full + s), C::KVB + (tensor ? 16u * pages : 0u));
                    __syncwarp();
                    if (lane < C::NH)
                        tma_load_3d((tensor ? v_s(s) : k_s(s)) + lane * C::HALF, tensor ? &tm_v : &tm_k, lane * 64,
                                    tile.kv_head, at * kBlockSize, bar(full + s));
                    else if (tensor && lane == C::NH)
                        bulk_load(f_s(s, 0), sp.factors + static_cast<int64_t>(tile.kv_head) * p.num_blocks + at,
                                  16u * pages, bar(full + s));
                    ++issued[tensor];
                }
                if (!ok) break;
            }
        }
        if (lane == 0) {
            // no TMA write may outlive the CTA
            if (n_q_loads > 0 && !mbar_wait(bar(B_QFULL), (n_q_loads - 1) & 1, nullptr)) atomicOr(p.err, kErrTimeout);
            for (int tensor = 0; tensor < 2; ++tensor) {
                const int ns = tensor ? C::NSV : C::NSK;
                for (int k = issued[tensor] - 1; k >= 0 && k >= issued[tensor] - ns; --k) {
                    const int s = k % ns, n = k / ns;
                    if (!mbar_wait(bar((tensor ? B_VFULL : B_KFULL) + s), n & 1, nullptr))
                        atomicOr(p.err, kErrTimeout);
                }
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------------ MMA issuer --
        issue_mmas<D, C, SPLIT>(p, smem_u32(bars), q_s(0), k_s(0), v_s(0), tmem, tile_begin, tile_end, tpt, lane, &abort_flag);
      }
    } else {
        // ------------------------------------------- softmax + epilogue --
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::REGS_SOFTMAX));
        const int t = (warp - 4) / 4;            // sub-tile of this warpgroup
        const int quarter = warp & 3;            // tensor-memory lanes 32*quarter .. +31
        const int row = quarter * 32 + lane;
        const uint32_t t_row = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
        int scnt = 0, ocnt = 0;                  // S tiles and outputs consumed by this sub-tile
        int n_split = 0;                         // split tiles so far
        int vbase = 0;                           // V tiles of the previous tiles of this CTA
        int v_seen = 0;                          // one past the last V tile waited for
        bool ok = true;
        for (int ti = tile_begin; ti < tile_end && ok; ++ti) {
            const ExtendTile tile = p.tiles[p.cta_tiles[ti]];
            const TileShape sh = tile_shape<SPLIT>(tile, tpt);
            const int i = (sh.split ? 0 : t * tpt) + row / G;   // token of this row within the tile
            const int gq = row % G;
            // rows past tpt * G (when G does not divide 128) are padding
            const bool tok_valid = row < tpt * G && i < tile.n_tok;
            const int pos_lim = tile.causal ? tile.pos0 + i + 1 : 0x7fffffff;  // keys < pos_lim
            const int row_end = min(tile.key_end, pos_lim);
            const int n_mine = t ? sh.n_sub[1] : sh.n_sub[0];
            // windows: this row's begins at low, the tile's first one at low_min
            const int low = pos_lim - p.window, low_min = tile.pos0 + 1 - p.window;
            float m = -INFINITY, l = 0.f;
            for (int i_step = 0; i_step < n_mine; ++i_step) {
                const int j = sh.step(i_step, t);   // key tile
                const int kt0 = tile.key_begin + j * kTileKeys;
                // Behind tiles whose empty second sub-tile passed this warpgroup by,
                // S comes first: the parity of a V barrier tells two neighbouring
                // phases apart only, and this warpgroup has not seen the phase
                // before the one asked for (nor has it of a split tile, whose key tiles it
                // sees every second of).  S completes behind every MMA of the key tiles
                // before, so that phase is over.  (S first in every tile:
                // 214.0 us instead of 212.8 for the two chunks above.)
                const bool s_first = sh.split || vbase + j >= v_seen + C::NSV;
                if (s_first && !warp_wait(bar(B_SFULL + t), scnt & 1, &abort_flag)) { ok = false; break; }
                v_seen = vbase + j + 1;
                // the factors of the tile's blocks, which came with its V stage,
                // while S is being computed; blocks past the key range have none,
                // and masked columns
                const int vs_stage = (vbase + j) % C::NSV;
                if (!warp_wait(bar(B_VFULL + vs_stage), ((vbase + j) / C::NSV) & 1, &abort_flag)) { ok = false; break; }
                float fs[8], lv[8], iv[8];
#pragma unroll
                for (int b = 0; b < 8; ++b) {
                    const uint4 f = lds_v4(f_s(vs_stage, b));
                    fs[b] = __uint_as_float(f.x);
                    lv[b] = __uint_as_float(f.y);
                    iv[b] = __uint_as_float(f.z);
                }
                if (tile.key_end - kt0 < kTileKeys) {
#pragma unroll
                    for (int b = 0; b < 8; ++b)
                        if (kt0 + kBlockSize * b >= tile.key_end) { fs[b] = 1.f; lv[b] = 0.f; iv[b] = 0.f; }
                }
                // blocks without a key that some row of the tile sees (the head's
                // padding, which has no factors, among them)
                const bool behind = WIN && kt0 < low_min && kt0 + kTileKeys > p.sinks;
                if (behind) {
#pragma unroll
                    for (int b = 0; b < 8; ++b)
                        if (kt0 + kBlockSize * b >= p.sinks && kt0 + kBlockSize * (b + 1) <= low_min) {
                            fs[b] = 1.f; lv[b] = 0.f; iv[b] = 0.f;
                        }
                }
                if (!s_first && !warp_wait(bar(B_SFULL + t), scnt & 1, &abort_flag)) { ok = false; break; }
                ++scnt;
                tc_fence_after();
                const int lim = row_end - kt0;       // columns < lim are visible
                // the whole S row in registers: four loads, one wait
                uint32_t sr[128];
                tmem_ld32(t_row + col_s(t) + 0, *reinterpret_cast<uint32_t(*)[32]>(&sr[0]));
                tmem_ld32(t_row + col_s(t) + 32, *reinterpret_cast<uint32_t(*)[32]>(&sr[32]));
                tmem_ld32(t_row + col_s(t) + 64, *reinterpret_cast<uint32_t(*)[32]>(&sr[64]));
                tmem_ld32(t_row + col_s(t) + 96, *reinterpret_cast<uint32_t(*)[32]>(&sr[96]));
                tmem_wait_ld();
                // keys past the row's limit, or behind its window and not first tokens
                if (lim < kTileKeys || (WIN && kt0 < low)) {
                    const int from = p.sinks - kt0, to = low - kt0;
                    hide_columns<WIN>(sr, lim, from, to);
#pragma unroll
                    for (int b = 0; b < 8; ++b)   // none of the block: its scale, NaN even, plays no part
                        if (kBlockSize * b >= lim || (WIN && kBlockSize * b >= from && kBlockSize * (b + 1) <= to)) fs[b] = 1.f;
                }
                // row max of s + log2 vs
                float mxs = -INFINITY;
#pragma unroll
                for (int b = 0; b < 8; ++b) {
                    auto s = [&](int c) { return __uint_as_float(sr[16 * b + c]); };
                    float mx0 = max3(s(0), s(1), s(2)), mx1 = max3(s(3), s(4), s(5));
                    mx0 = max3(mx0, s(6), s(7));
                    mx1 = max3(mx1, s(8), s(9));
                    mx0 = max3(mx0, s(10), s(11));
                    mx1 = max3(mx1, s(12), s(13));
                    mx0 = max3(mx0, s(14), s(15));
                    mxs = fmaxf(mxs, fmaf(fmaxf(mx0, mx1), fs[b], lv[b]));
                }
                const bool need = mxs > m + 8.f;
                float alpha = 1.f;
                if (need) {
                    alpha = ex2(m - mxs);
                    m = mxs;
                    l *= alpha;
                }
                const float nref = m == -INFINITY ? 0.f : -m;
                // w = exp2(s + log2 vs - m) as f16 pairs, packed in place (entry e
                // takes columns 2e and 2e+1, which are read before entry e is
                // written), then stored over the first 64 columns of S; the
                // scale-and-shift and the sums run on packed fp32 pairs
                uint64_t l2 = f32x2(0.f, 0.f);
#pragma unroll
                for (int b = 0; b < 8; ++b) {
                    const uint64_t scale2 = f32x2(fs[b], fs[b]), shift2 = f32x2(lv[b] + nref, lv[b] + nref);
                    uint64_t w[2];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const int c = 16 * b + 2 * e;
                        float x0, x1;
                        f32x2_split(fma_f32x2(f32x2(__uint_as_float(sr[c]), __uint_as_float(sr[c + 1])), scale2, shift2),
                                    x0, x1);
                        const float p0 = ex2(x0), p1 = ex2(x1);
                        w[e & 1] = e < 2 ? f32x2(p0, p1) : add_f32x2(w[e & 1], f32x2(p0, p1));
                        sr[8 * b + e] = pack_f16x2(p0, p1);
                    }
                    l2 = fma_f32x2(add_f32x2(w[0], w[1]), f32x2(iv[b], iv[b]), l2);
                    if (b == 3) {   // the first half of P, under which its PV can begin
                        tmem_st32(t_row + col_s(t) + 0, *reinterpret_cast<uint32_t(*)[32]>(&sr[0]));
                        if (i_step >= 1 && __any_sync(0xffffffffu, need)) {
                            // O_t holds the key tiles before (their PV completed before S_t(j) did)
#pragma unroll 1
                            for (int c = 0; c < D; c += 32) {
                                uint32_t orr[32];
                                tmem_ld32(t_row + col_o(t) + c, orr);
                                tmem_wait_ld();
#pragma unroll
                                for (int e = 0; e < 32; ++e) orr[e] = __float_as_uint(__uint_as_float(orr[e]) * alpha);
                                tmem_st32(t_row + col_o(t) + c, orr);
                            }
                        }
                        tmem_wait_st();
                        // value rows past the end of the key range may hold anything
                        // (unwritten slots, stale blocks, NaN): zero them so that
                        // 0 * row stays 0 inside the MMA.  Each sub-tile that reads
                        // the last V tile zeroes them before handing over its P, so
                        // the PV after it sees zeros (both write the same zeros).  So
                        // it is for rows that no window of the tile reaches and that
                        // are not first tokens.
                        const int valid_keys = tile.key_end - kt0;
                        if ((valid_keys < kTileKeys && j == sh.n_tiles - 1) || behind) {
                            const int s = vs_stage;   // (landed: waited for above)
                            if (row >= valid_keys || (behind && kt0 + row >= p.sinks && kt0 + row < low_min)) {
#pragma unroll
                                for (int h = 0; h < C::NH; ++h)
#pragma unroll
                                    for (int ch = 0; ch < 8; ++ch) {
                                        const uint32_t a = v_s(s) + h * C::HALF + row * 128 + ch * 16;
                                        asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(a), "r"(0) : "memory");
                                    }
                            }
                            fence_proxy_async_smem();
                        }
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(bar(B_PFULL + t));
                    }
                }
                float l0, l1;
                f32x2_split(l2, l0, l1);
                l += l0 + l1;
                tmem_st32(t_row + col_s(t) + 32, *reinterpret_cast<uint32_t(*)[32]>(&sr[32]));
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(B_PFULL + 2 + t));
            }
            if (!ok) break;
            vbase += sh.n_tiles;
            // ------------------------------------------------- epilogue --
            if (n_mine == 0) continue;
            if (!warp_wait(bar(B_ODONE + t), ocnt & 1, &abort_flag)) { ok = false; break; }
            ++ocnt;
            tc_fence_after();
            // a split tile: sub-tile 1 hands over its maximum and sum, and goes on when
            // sub-tile 0 has read its O
            Joined joined;
            if (sh.split) {
                if (t == 1) {
                    second[row] = make_float2(m, l);
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(B_SECOND));
                    if (!warp_wait(bar(B_JOINED), n_split & 1, &abort_flag)) { ok = false; break; }
                    ++n_split;
                    tc_fence_after();
                    continue;
                }
                if (!warp_wait(bar(B_SECOND), n_split & 1, &abort_flag)) { ok = false; break; }
                ++n_split;
                tc_fence_after();
                joined.join(m, l, second[row]);
            }
            const float inv = l == 0.f ? 0.f : 1.f / l;   // no visible key: 0; a NaN stays one
            const int tok = tile.t0 + i;
            const int h = tile.kv_head * G + gq;
            int64_t slot = -1;
            if (tile.part >= 0 && tok_valid)
                slot = static_cast<int64_t>(p.part_offset[tok * p.n_groups + tile.kv_head / p.heads_per_group]) +
                       tile.part;
            store_output<D>(p, t_row + col_o(t), t_row + col_o(1), sh.split, tok_valid, tile.part, tok, h, slot,
                            joined.a0 * inv, joined.a1 * inv, lane, [&] {
                                if (!sh.split) return;
                                tc_fence_before();
                                __syncwarp();
                                if (lane == 0) mbar_arrive(bar(B_JOINED));
                            });
            // the partial's weight 2^m l in the merge, kept as l = 1 (L holds the
            // range of 1 / vs); a NaN takes the merge over
            if (tok_valid && tile.part >= 0)
                p.ml_part[slot * p.num_heads_q + h] =
                    l == 0.f ? make_float2(-INFINITY, 0.f) : make_float2(l != l ? 3.0e38f : m + lg2(l), 1.f);
            tc_fence_before();
        }
        if (!ok) raise_abort(&abort_flag, p.err, kErrTimeout);
    }
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, C::TMEM_COLS);
    }
}

template <int D, bool WIN, bool SPLIT>
cudaError_t configure() {
    // the attribute is per function and device; setting it again is harmless
    return cudaFuncSetAttribute(scaled_extend_kernel<D, WIN, SPLIT>, cudaFuncAttributeMaxDynamicSharedMemorySize, ScaledExtCfg<D>::SMEM);
}

template <int D, bool WIN, bool SPLIT>
cudaError_t launch_t(int grid, const CUtensorMap &tm_q, const CUtensorMap &tm_k, const CUtensorMap &tm_v,
                     const ScaledExtendParams &p, cudaStream_t stream, bool pdl) {
    using C = ScaledExtCfg<D>;
    return launch_ex(scaled_extend_kernel<D, WIN, SPLIT>, dim3(grid), dim3(C::THREADS), C::SMEM, stream, pdl, tm_q, tm_k, tm_v, p);
}

}  // namespace

#define PA_EXTEND_CASE(window, split, f, ...)                                                     \
    if (head_dim == 128)                                                                          \
        return !(window) ? f<128, false, false>(__VA_ARGS__)                                      \
               : (split) ? f<128, true, true>(__VA_ARGS__) : f<128, true, false>(__VA_ARGS__);    \
    if (head_dim == 64)                                                                           \
        return !(window) ? f<64, false, false>(__VA_ARGS__)                                       \
               : (split) ? f<64, true, true>(__VA_ARGS__) : f<64, true, false>(__VA_ARGS__);      \
    return cudaErrorInvalidValue;

cudaError_t prepare_scaled_extend(int head_dim, bool window, bool split) { PA_EXTEND_CASE(window, split, configure) }

cudaError_t launch_scaled_extend(int head_dim, int grid, const CUtensorMap &tm_q, const CUtensorMap &tm_k,
                          const CUtensorMap &tm_v, const ScaledExtendParams &p, cudaStream_t stream, bool pdl) {
    if (grid <= 0) return cudaSuccess;
    PA_EXTEND_CASE(p.base.window > 0, p.base.split != 0, launch_t, grid, tm_q, tm_k, tm_v, p, stream, pdl)
}
#undef PA_EXTEND_CASE

}  // namespace pa
