// Extend / chunked-prefill attention on the 5th-generation tensor cores
// (tcgen05, accumulators in tensor memory), and the shared-prefix stage of
// the cascade route.
//
// What one CTA computes (page "vLLM 推理流程分析" §6.2: varlen causal
// attention through block_table; §10.1: a token sees itself and earlier
// tokens; §5.1.2: positions = num_computed + offset in the chunk):
//   up to 256 query rows = 2 sub-tiles of 128 rows, each 128/G consecutive
//   tokens x the G query heads of one kv head, against keys
//   [key_begin, key_end) of one request's context, read through the block
//   table in tiles of 128 keys (8 blocks).  Row (i, g) at absolute position
//   pos0 + i sees key j iff j <= pos0 + i (causal tiles); shared-prefix tiles
//   see their whole key range.  Both sub-tiles share every K/V tile loaded.
//
// Per 128-key tile and sub-tile t:
//   S_t = Q_t K^T        tcgen05.mma M=128 N=128 K=D, A and B from shared memory
//   P_t = exp2(S_t*scale*log2e - m)   softmax warpgroup t, one row per thread,
//                        written back to tensor memory over S_t as bf16 pairs
//   O_t += P_t V         tcgen05.mma M=128 N=D K=128, A from tensor memory
// Warp roles: warp 0 TMA producer (Q once, K and V blocks into 2- and 3-stage
// rings; a V stage is released as soon as both PVs reading it are done),
// warp 1 MMA issuer and tensor-memory owner (issue_mmas), warps 2-3 idle but for
// split tiles' V (warpgroup 0 gives its registers to the softmax warpgroups), warps
// 4-7 softmax of sub-tile 0, warps 8-11 softmax of sub-tile 1.  The issuer
// alternates between the sub-tiles, so the tensor core works on one while the
// other's softmax runs.  The running max only moves (and O is rescaled) when it
// grows by more than 2^8, which keeps every weight <= 256.
//
// Two chunks of 2048 tokens over 0 and 4096 (Hq 32, Hkv 8, D 128): 138 us, 1497
// TFLOP/s; over a window of 1024 with 4 first tokens: 69 us, 1000 TFLOP/s of what is
// seen.  There a tile has 9 steps: 512 tiles on 152 SMs are four rounds of 3.4 (16%),
// 11% of a tile's columns are hidden ones, their masks take 2.5 us, the epilogue 3, and
// the tensor pipe is active for 45%.
//
// Tensor memory (512 columns x 128 lanes, fp32): S_0 [0,128), S_1 [128,256)
// (P_t in the first 64 columns of S_t), O_0 [256,256+D), O_1 [384,384+D).
// Shared memory tiles are 128-byte-swizzled [rows][64 elements] halves:
// Q_t (A, K-major), K (B, K-major), V (B, MN-major).
#include <atomic>

#include "tiles.cuh"

namespace pa {
namespace {

using namespace dev;
using namespace tiles;

template <int D>
struct ExtCfg {
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
    static constexpr int TILE_SMEM = 2 * QB + (NSK + NSV) * KVB;
    // one CTA per SM: it owns all 512 tensor-memory columns
    static constexpr int SMEM = (TILE_SMEM + 1024 < 120 * 1024) ? 120 * 1024 : TILE_SMEM + 1024;
    static constexpr uint32_t TMEM_COLS = 512;
    static constexpr uint32_t IDESC_QK = idesc_bf16(128, 128, false, false);
    static constexpr uint32_t IDESC_PV = idesc_bf16(128, D, false, true);
};


// WIN: with a sliding window and first tokens (tiles in WindowView's numbers: key
// tiles of 128 keys run over the blocks with first tokens and on into those of the
// tile's first window, whose lower masks reach over the first key tiles only).
// SPLIT (with a window): some or all of the tiles are of one sub-tile of rows whose keys
// both sub-tiles share (variants of their own: kSomeSplit costs the other tiles 3%, and
// 512 tokens over 4096 keys 41.1 us instead of kAllSplit's 37.1).  Sharing
// doubles the loads per step: K and V in boxes of one block and 64 columns (2 KB) come
// at 46 GB/s per SM (the TMA unit's time per box), which that needs twice of.  So V
// of such tiles comes by 16-byte asynchronous copies of the two idle warps (a step of
// two key tiles 1.7 us instead of 2.8; in the other tiles they would cost 6%, by the
// issue slots they take).  The planner splits all tiles of a step over bf16 caches or
// none, so that one side brings every V tile of a CTA.  COPIES: over the consecutive
// 16-bit copies of E4M3 blocks, a key tile is one box per 64 columns.
template <int D, bool WIN, bool COPIES, int SPLIT>
__global__ void __launch_bounds__(384, 1)
extend_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
              const __grid_constant__ CUtensorMap tm_v, const ExtendParams p) {
    using C = ExtCfg<D>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ int abort_flag;
    __shared__ uint32_t tmem_base_slot;
    __shared__ __align__(8) uint64_t bars[NUM_BARS];
    __shared__ float2 second[SPLIT != 0 ? kTileRows : 1];   // split tiles: sub-tile 1's maximum and sum of each row

    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    auto q_s = [&](int t) { return base + static_cast<uint32_t>(t) * C::QB; };
    auto k_s = [&](int s) { return base + 2 * C::QB + static_cast<uint32_t>(s) * C::KVB; };
    auto v_s = [&](int s) { return base + 2 * C::QB + static_cast<uint32_t>(C::NSK + s) * C::KVB; };
    auto bar = [&](int i) { return smem_u32(&bars[i]); };

    grid_launch_dependents();
    grid_dep_wait();    // the work list and caches come from earlier kernels of the stream
    // this CTA's tiles, longest first (the planner's greedy assignment)
    const int tile_begin = p.cta_tile_begin[blockIdx.x];
    const int tile_end = p.cta_tile_begin[blockIdx.x + 1];
    if (tile_begin >= tile_end) return;
    // warps 2 and 3 bring V
    const bool v_warps = !COPIES && (SPLIT == kAllSplit || (SPLIT == kSomeSplit && p.tiles[p.cta_tiles[tile_begin]].split != 0));
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
            mbar_init(bar(B_VFULL + s), v_warps ? 2 : 1);
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
            const TileShape sh = tile_shape<SPLIT != 0>(tile, tpt);
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
            const int32_t *bt = p.block_table + static_cast<int64_t>(tile.req) * p.max_blocks;
            if constexpr (COPIES) {
                // the copies of the head (rows of its padding are other blocks'), then
                // those from page `head` on, counted from the tile's first page
                const int pg_begin = tile.key_begin / kBlockSize, head = tile.head - pg_begin;
                const int pg_end = (tile.key_end - tile.key_begin + kBlockSize - 1) / kBlockSize;
                const int32_t dst0 = bt[tile.head + tile.skip] - head, head0 = head > 0 ? bt[0] + pg_begin : 0;
                if (dst0 + max(head, 0) < 0 || dst0 + pg_end > p.num_blocks || head0 < 0) {   // (not from the planner)
                    if (lane == 0) raise_abort(&abort_flag, p.err, kErrBlockRange);
                    break;
                }
                for (int j = 0; j < sh.n_tiles && ok; ++j) {
                    const int pg0 = j * (kTileKeys / kBlockSize);
                    const int32_t at = (pg0 < head ? head0 : dst0) + pg0;
#pragma unroll
                    for (int tensor = 0; tensor < 2; ++tensor) {
                        const int ns = tensor ? C::NSV : C::NSK;
                        const int s = issued[tensor] % ns, n = issued[tensor] / ns;
                        const int full = tensor ? B_VFULL : B_KFULL;
                        if (n > 0 && !warp_wait(bar((tensor ? B_VEMPTY : B_KEMPTY) + s), (n & 1) ^ 1, &abort_flag)) {
                            if (lane == 0) raise_abort(&abort_flag, p.err, kErrTimeout);
                            ok = false;
                            break;
                        }
                        if (lane == 0) mbar_arrive_expect_tx(bar(full + s), C::KVB);
                        __syncwarp();
                        if (lane < C::NH)
                            tma_load_3d((tensor ? v_s(s) : k_s(s)) + lane * C::HALF, tensor ? &tm_v : &tm_k, lane * 64,
                                        tile.kv_head, at * kBlockSize, bar(full + s));
                        ++issued[tensor];
                    }
                }
                continue;
            }
            // block ids of 32 pages (4 key tiles) per load: the producer's
            // dependent block-table read happens once per window, not per tile
            const int pg_end = (tile.key_end + kBlockSize - 1) / kBlockSize;
            int32_t win = 0;
            int win0 = -64;
            for (int j = 0; j < sh.n_tiles; ++j) {
                const int kt0 = tile.key_begin + j * kTileKeys;
                const int pg0 = kt0 / kBlockSize;
                const int pages = min(8, (tile.key_end - kt0 + kBlockSize - 1) / kBlockSize);
                if (pg0 + 8 > win0 + 32) {
                    win0 = pg0;
                    const int pg = WIN ? WindowView{tile.head, tile.skip}.at(pg0 + lane) : pg0 + lane;
                    win = pg0 + lane < pg_end ? bt[pg] : 0;
                }
                const int32_t mine_blk = __shfl_sync(0xffffffffu, win, (pg0 - win0 + (lane & 7)) & 31);
                int32_t blk = 0;
                bool valid = false;
                if (lane < pages) {
                    blk = mine_blk;
                    valid = blk >= 0 && blk < p.num_blocks;
                }
                const unsigned vmask = __ballot_sync(0xffffffffu, valid);
                const uint32_t bytes = __popc(vmask) * kBlockSize * 128 * C::NH;
                if (lane == 0 && __popc(vmask) != pages) atomicOr(p.err, kErrBlockRange);
                static_assert(8 * C::NH <= 32, "one TMA box per lane");
                const int page = lane / C::NH;
                const int half = lane % C::NH;
                const int32_t b = __shfl_sync(0xffffffffu, blk, page & 7);  // every lane takes part
                const bool mine = lane < 8 * C::NH && ((vmask >> page) & 1u);
#pragma unroll
                for (int tensor = 0; tensor < 2; ++tensor) {
                    if (tensor && v_warps) continue;
                    const int ns = tensor ? C::NSV : C::NSK;
                    const int s = issued[tensor] % ns, n = issued[tensor] / ns;
                    const int empty = tensor ? B_VEMPTY : B_KEMPTY;
                    const int full = tensor ? B_VFULL : B_KFULL;
                    if (n > 0 && !warp_wait(bar(empty + s), (n & 1) ^ 1, &abort_flag)) {
                        if (lane == 0) raise_abort(&abort_flag, p.err, kErrTimeout);
                        ok = false;
                        break;
                    }
                    if (lane == 0) mbar_arrive_expect_tx(bar(full + s), bytes);
                    __syncwarp();
                    if (mine)
                        tma_load_3d((tensor ? v_s(s) : k_s(s)) + half * C::HALF + page * 2048,
                                    tensor ? &tm_v : &tm_k, half * 64, tile.kv_head, b * kBlockSize, bar(full + s));
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
        issue_mmas<D, C, SPLIT != 0>(p, smem_u32(bars), q_s(0), k_s(0), v_s(0), tmem, tile_begin, tile_end, tpt, lane, &abort_flag);
      } else if (v_warps) {
        // ------------------------------------------------------- V copies --
        // Each warp brings 64 rows (4 blocks) of a V tile, swizzled as a box would
        // be, and hands them over a tile later, so that its copies are under way
        // while it waits for the next stage.
        constexpr int CH = D / 8;                // 16-byte chunks of a row
        const int64_t row_elems = static_cast<int64_t>(p.num_heads_kv) * D;
        int issued = 0;
        bool ok = true;
        auto hand_over = [&](int i) {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(B_VFULL + i % C::NSV));
        };
        for (int ti = tile_begin; ti < tile_end && ok; ++ti) {
            const ExtendTile tile = p.tiles[p.cta_tiles[ti]];
            const TileShape sh = tile_shape<SPLIT != 0>(tile, tpt);
            const WindowView view{tile.head, tile.skip};
            const int32_t *bt = p.block_table + static_cast<int64_t>(tile.req) * p.max_blocks;
            const int pg_end = (tile.key_end + kBlockSize - 1) / kBlockSize;
            int32_t win = 0;                     // block ids of 32 pages
            int win0 = -64;
            for (int j = 0; j < sh.n_tiles; ++j) {
                const int pg0 = (tile.key_begin + j * kTileKeys) / kBlockSize;
                if (pg0 + 8 > win0 + 32) {
                    win0 = pg0;
                    win = pg0 + lane < pg_end ? bt[view.at(pg0 + lane)] : -1;
                }
                const int s = issued % C::NSV, n = issued / C::NSV;
                if (n > 0 && !warp_wait(bar(B_VEMPTY + s), (n & 1) ^ 1, &abort_flag)) {
                    if (lane == 0) raise_abort(&abort_flag, p.err, kErrTimeout);
                    ok = false;
                    break;
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int page = 4 * (warp - 2) + k;
                    const int32_t blk = __shfl_sync(0xffffffffu, win, (pg0 - win0 + page) & 31);
                    if (pg0 + page >= pg_end || blk < 0 || blk >= p.num_blocks) continue;   // (reported with K)
                    const uint16_t *src = p.value_cache + blk * kBlockSize * row_elems + tile.kv_head * D;
#pragma unroll
                    for (int i = 0; i < kBlockSize * CH / 32; ++i) {
                        const int row = (32 * i + lane) / CH, c = (32 * i + lane) % CH;
                        cp_async16(v_s(s) + (c / 8) * C::HALF + (page * kBlockSize + row) * 128 + (((c % 8) ^ (row & 7)) << 4),
                                   src + row * row_elems + c * 8);
                    }
                }
                cp_async_commit();
                if (issued > 0) {
                    cp_async_wait<1>();
                    hand_over(issued - 1);
                }
                ++issued;
            }
        }
        // no copy may outlive the CTA
        cp_async_wait_all();
        if (issued > 0) hand_over(issued - 1);
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
        bool ok = true;
        for (int ti = tile_begin; ti < tile_end && ok; ++ti) {
            const ExtendTile tile = p.tiles[p.cta_tiles[ti]];
            const TileShape sh = tile_shape<SPLIT != 0>(tile, tpt);
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
                if (!warp_wait(bar(B_SFULL + t), scnt & 1, &abort_flag)) { ok = false; break; }
                ++scnt;
                tc_fence_after();
                const int kt0 = tile.key_begin + j * kTileKeys;
                const int lim = row_end - kt0;       // columns < lim are visible
                // the whole S row in registers: four loads, one wait
                uint32_t sr[128];
                tmem_ld32(t_row + col_s(t) + 0, *reinterpret_cast<uint32_t(*)[32]>(&sr[0]));
                tmem_ld32(t_row + col_s(t) + 32, *reinterpret_cast<uint32_t(*)[32]>(&sr[32]));
                tmem_ld32(t_row + col_s(t) + 64, *reinterpret_cast<uint32_t(*)[32]>(&sr[64]));
                tmem_ld32(t_row + col_s(t) + 96, *reinterpret_cast<uint32_t(*)[32]>(&sr[96]));
                tmem_wait_ld();
                // keys past the row's limit, or behind its window and not first tokens
                if (lim < kTileKeys || (WIN && kt0 < low)) hide_columns<WIN>(sr, lim, p.sinks - kt0, low - kt0);
                // row max: 3-input max, four chains
                float mx0 = -INFINITY, mx1 = -INFINITY, mx2 = -INFINITY, mx3 = -INFINITY;
#pragma unroll
                for (int c = 0; c < 128; c += 8) {
                    mx0 = max3(mx0, __uint_as_float(sr[c]), __uint_as_float(sr[c + 1]));
                    mx1 = max3(mx1, __uint_as_float(sr[c + 2]), __uint_as_float(sr[c + 3]));
                    mx2 = max3(mx2, __uint_as_float(sr[c + 4]), __uint_as_float(sr[c + 5]));
                    mx3 = max3(mx3, __uint_as_float(sr[c + 6]), __uint_as_float(sr[c + 7]));
                }
                const float mxs = fmaxf(fmaxf(mx0, mx1), fmaxf(mx2, mx3)) * p.scale_log2;
                const bool need = mxs > m + 8.f;
                float alpha = 1.f;
                if (need) {
                    alpha = ex2(m - mxs);
                    m = mxs;
                    l *= alpha;
                }
                const float nref = m == -INFINITY ? 0.f : -m;
                // P = exp2(s*scale - m) as bf16 pairs, packed in place (entry e
                // takes columns 2e and 2e+1, which are read before entry e is
                // written), then stored over the first 64 columns of S; the
                // scale-and-shift and the row sum run on packed fp32 pairs
                const uint64_t scale2 = f32x2(p.scale_log2, p.scale_log2), shift2 = f32x2(nref, nref);
                uint64_t la = f32x2(0.f, 0.f), lb = la;
                auto weights = [&](int from) {   // 64 columns from there on
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        const int e = from / 2 + i;
                        float x0, x1;
                        f32x2_split(fma_f32x2(f32x2(__uint_as_float(sr[2 * e]), __uint_as_float(sr[2 * e + 1])), scale2,
                                              shift2),
                                    x0, x1);
                        const float p0 = ex2(x0), p1 = ex2(x1);
                        if (e & 1) lb = add_f32x2(lb, f32x2(p0, p1));
                        else la = add_f32x2(la, f32x2(p0, p1));
                        sr[e] = pack_bf16x2(p0, p1);
                    }
                    tmem_st32(t_row + col_s(t) + from / 2, *reinterpret_cast<uint32_t(*)[32]>(&sr[from / 2]));
                };
                // the first half of P, under which its PV can begin
                weights(0);
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
                // the PV after it sees zeros (both write the same zeros).  So it is
                // for rows that no window of the tile reaches and that are not
                // first tokens.  (V tiles before this one are full: S_t(j) stands
                // behind the PVs of theirs.)
                const int valid_keys = tile.key_end - kt0;
                const bool behind = WIN && kt0 < low_min && kt0 + kTileKeys > p.sinks;
                if ((valid_keys < kTileKeys && j == sh.n_tiles - 1) || behind) {
                    const int vi = vbase + j;
                    const int s = vi % C::NSV;
                    if (!warp_wait(bar(B_VFULL + s), (vi / C::NSV) & 1, &abort_flag)) { ok = false; break; }
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
                weights(64);
                float a0, a1, b0, b1;
                f32x2_split(la, a0, a1);
                f32x2_split(lb, b0, b1);
                l += (a0 + b0) + (a1 + b1);
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
            const float inv = l > 0.f ? p.out_scale / l : 0.f;
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
            if (tok_valid && tile.part >= 0) p.ml_part[slot * p.num_heads_q + h] = partial_weight(m, l);
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

template <int D, bool WIN, bool COPIES, int SPLIT>
cudaError_t configure() {
    // the attribute is per function and device: set once for each
    static std::atomic<uint64_t> configured{0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!(configured.load(std::memory_order_relaxed) >> dev & 1)) {
        cudaError_t e = cudaFuncSetAttribute(extend_kernel<D, WIN, COPIES, SPLIT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             ExtCfg<D>::SMEM);
        if (e != cudaSuccess) return e;
        configured.fetch_or(uint64_t{1} << dev, std::memory_order_relaxed);
    }
    return cudaSuccess;
}

template <int D, bool WIN, bool COPIES, int SPLIT>
cudaError_t launch_t(int grid, const CUtensorMap &tm_q, const CUtensorMap &tm_k, const CUtensorMap &tm_v,
                     const ExtendParams &p, cudaStream_t stream, bool pdl) {
    using C = ExtCfg<D>;
    cudaError_t e = configure<D, WIN, COPIES, SPLIT>();
    if (e != cudaSuccess) return e;
    return launch_ex(extend_kernel<D, WIN, COPIES, SPLIT>, dim3(grid), dim3(C::THREADS), C::SMEM, stream, pdl, tm_q, tm_k, tm_v, p);
}

}  // namespace

// f<D, WIN, COPIES, SPLIT> of a plan's variant (E4M3 caches, whose tiles read copies, have
// head_dim 128)
#define PA_EXTEND_SPLIT(d, copies, split, f, ...)                                 \
    return (split) == kNoSplit     ? f<d, true, copies, kNoSplit>(__VA_ARGS__)    \
           : copies || (split) == kSomeSplit ? f<d, true, copies, kSomeSplit>(__VA_ARGS__) \
                                   : f<d, true, copies, copies ? kSomeSplit : kAllSplit>(__VA_ARGS__);
#define PA_EXTEND_CASE(window, copies, split, f, ...)                                  \
    if (head_dim == 128 && !(window)) return f<128, false, false, kNoSplit>(__VA_ARGS__); \
    if (head_dim == 64 && !(window)) return f<64, false, false, kNoSplit>(__VA_ARGS__);   \
    if (head_dim == 128 && (copies)) PA_EXTEND_SPLIT(128, true, split, f, __VA_ARGS__)    \
    if (head_dim == 128) PA_EXTEND_SPLIT(128, false, split, f, __VA_ARGS__)               \
    if (head_dim == 64) PA_EXTEND_SPLIT(64, false, split, f, __VA_ARGS__)                 \
    return cudaErrorInvalidValue;

cudaError_t prepare_extend(int head_dim, bool window, bool copies, int split) {
    PA_EXTEND_CASE(window, copies, split, configure)
}

cudaError_t launch_extend(int head_dim, int grid, const CUtensorMap &tm_q, const CUtensorMap &tm_k,
                          const CUtensorMap &tm_v, const ExtendParams &p, cudaStream_t stream, bool pdl) {
    if (grid <= 0) return cudaSuccess;
    PA_EXTEND_CASE(p.window > 0, p.value_cache == nullptr, p.split, launch_t, grid, tm_q, tm_k, tm_v, p, stream, pdl)
}
#undef PA_EXTEND_CASE
#undef PA_EXTEND_SPLIT

}  // namespace pa
